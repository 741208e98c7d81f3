"""Device-buffer plumbing around the C ABI for one BitLinear weight.

`BitLinearWeight` owns the device buffers of one layer (mask, packed codes,
gamma, workspaces) and calls the library's entry points in the order the
method runs them: quantize_mask + pack once per training step (the mask is
recomputed every step) or once at load time for inference, then fwd / bwd
per batch.  torch is used for device memory and the stream only.
"""
import numpy as np
import torch

from . import bitlinear as bl


def bf16_tensor(bits: np.ndarray, device="cuda") -> torch.Tensor:
    """uint16 bf16 bit patterns (numpy) -> torch.bfloat16 device tensor."""
    t = torch.from_numpy(np.ascontiguousarray(bits, dtype=np.uint16).view(np.int16))
    return t.view(torch.bfloat16).to(device)


def bf16_bits(t: torch.Tensor) -> np.ndarray:
    return t.detach().contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


class BitLinearWeight:
    def __init__(self, n_out, k, n=6, m=8, gamma_over=bl.BL_GAMMA_DENSE, device="cuda"):
        self.n_out, self.k, self.n, self.m = int(n_out), int(k), int(n), int(m)
        self.gamma_over = gamma_over
        nbytes = bl.bitlinear_packed_bytes(n_out, k, n, m)
        if nbytes == 0:
            raise ValueError(f"unsupported layer {n_out}x{k} {n}:{m}")
        self.mask = torch.empty(n_out * (k // 8), dtype=torch.uint8, device=device)
        self.packed = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.gamma = torch.empty(1, dtype=torch.float64, device=device)
        self.ws = torch.empty(bl.bitlinear_workspace_bytes(n_out, k), dtype=torch.uint8, device=device)
        self.device = device

    def quantize(self, W, wq=None, stream=None):
        """Mask + gamma (+ optional int8 codes), then pack."""
        bl.bitlinear_quantize_mask(W, self.n_out, self.k, self.n, self.m, self.gamma_over, self.mask,
                                   wq, self.gamma, self.ws, stream=stream)
        bl.bitlinear_pack(W, self.mask, self.gamma, self.n_out, self.k, self.n, self.m, self.packed,
                          stream=stream)

    def fwd_buffers(self, tokens):
        d = self.device
        ws_n = bl.bitlinear_fwd_workspace_bytes(tokens, self.k, self.n_out)
        return {
            "Y": torch.empty(tokens * self.n_out, dtype=torch.float32, device=d),
            "xq": torch.empty(tokens * self.k, dtype=torch.int8, device=d),
            "x_scale": torch.empty(max(tokens, 1), dtype=torch.float32, device=d)[:tokens],
            # zero-filled once: bitlinear_contract needs zero counters on entry
            # and leaves them zero (bitlinear_fwd clears them itself)
            "ws": torch.zeros(ws_n, dtype=torch.uint8, device=d) if ws_n else None,
        }

    def fwd(self, X, tokens, bufs=None, acc=None, stream=None):
        b = bufs if bufs is not None else self.fwd_buffers(tokens)
        bl.bitlinear_fwd(X, tokens, self.k, self.packed, self.n_out, self.n, self.m, self.gamma,
                         b["Y"], b["xq"], b["x_scale"], acc=acc, ws=b["ws"], stream=stream)
        return b

    def bwd_workspace(self, tokens):
        """Device scratch of the backward (bf16 operands of its products)."""
        n = bl.bitlinear_bwd_workspace_bytes(tokens, self.k, self.n_out)
        return torch.empty(max(n, 1), dtype=torch.uint8, device=self.device)

    def bwd(self, dY, xq, x_scale, tokens, dX=True, dW=True, ws=None, stream=None):
        d = self.device
        gx = torch.empty(tokens * self.k, dtype=torch.float32, device=d) if dX else None
        gw = torch.empty(self.n_out * self.k, dtype=torch.float32, device=d) if dW else None
        if ws is None:
            ws = self.bwd_workspace(tokens)
        bl.bitlinear_bwd(dY, xq, x_scale, self.packed, self.gamma, tokens, self.k, self.n_out,
                         self.n, self.m, gx, gw, ws=ws, stream=stream)
        return gx, gw


class QuantGroup:
    """Grouped weight quantisation of several BitLinearWeight layers that
    share one N:M pattern and gamma mode: the plan (device descriptors) is
    built once for fixed (weight, layer) pairs, then each `run` recomputes
    every mask, gamma and packed block in three launches."""

    def __init__(self, pairs, stream=None):
        lws = [lw for lw, _ in pairs]
        if not lws:
            raise ValueError("QuantGroup needs at least one layer")
        n, m, go = lws[0].n, lws[0].m, lws[0].gamma_over
        if any((lw.n, lw.m, lw.gamma_over) != (n, m, go) for lw in lws):
            raise ValueError("all layers of a QuantGroup share n, m and gamma_over")
        self.n, self.m, self.gamma_over = n, m, go
        self.weights = [W for _, W in pairs]
        entries = [dict(W=W, mask=lw.mask, gamma=lw.gamma, packed=lw.packed, n_out=lw.n_out, k=lw.k)
                   for lw, W in pairs]
        self.items = bl.make_quant_items(entries, n, m)
        d = lws[0].device
        self.ws = torch.empty(max(bl.bitlinear_quant_group_workspace_bytes(self.items, len(entries)), 1),
                              dtype=torch.uint8, device=d)
        self.plan = torch.empty(bl.bitlinear_quant_group_plan_bytes(self.items, len(entries)),
                                dtype=torch.uint8, device=d)
        bl.bitlinear_quant_group_plan(self.items, len(entries), n, m, go, self.ws, self.plan, stream=stream)

    def run(self, stream=None):
        bl.bitlinear_quant_group(self.plan, self.n, self.m, self.gamma_over, stream=stream)


class LatentWeights:
    """binary32 latent weights of one layer and the bf16 copy the weight
    path reads; `update` applies one plain gradient step on the device."""

    def __init__(self, W_bf16, device="cuda"):
        self.W = W_bf16.contiguous().to(device)
        self.master = self.W.float().contiguous()

    def update(self, dW, lr, stream=None):
        bl.bitlinear_latent_update(self.master, dW, self.master.numel(), lr, self.W, stream=stream)


class BlockAttention:
    """What stands between a block's q, k, v BitLinears and its o BitLinear:
    head norms with the rotation, and causal attention over packed sequences
    (prompts and training) or over a paged cache (serving).  Owns the rotation
    table; outputs and workspaces are allocated per call on torch's current
    stream, as torch's own operators do.

    A packed batch may be padded: rows of no sequence come back as zeros from
    attend and attend_bwd, since whatever is further on sums over all tokens
    (rotate_bwd for the norms' weights, the BitLinears' dW).  A program whose
    sequences fill their rows may pass padded=False, which spares filling the
    outputs (8192 tokens, 20 + 5 heads of 128: 105 MB over both calls)."""

    def __init__(self, hq, hkv, d, max_pos, base=10000.0, q_weight=None, k_weight=None, eps=1e-6, scale=None,
                 device="cuda"):
        self.hq, self.hkv, self.d, self.eps = int(hq), int(hkv), int(d), float(eps)
        self.q_weight, self.k_weight = q_weight, k_weight
        self.scale = float(scale) if scale is not None else self.d ** -0.5
        self.device = device
        self.table = torch.empty(max_pos, self.d // 2, 2, dtype=torch.float32, device=device)
        bl.bitlinear_rope_table(max_pos, self.d, base, self.table)

    def _bf16(self, rows, heads, zeros=False):
        new = torch.zeros if zeros else torch.empty
        return new(rows, heads * self.d, dtype=torch.bfloat16, device=self.device)

    def _scratch(self, nbytes):
        return torch.empty(nbytes, dtype=torch.uint8, device=self.device) if nbytes else None

    def rotate(self, Q, K, V, pos, cache=None, slots=None):
        """(Qr, Kr, Vr) of the projections' rows; with a cache (K, V) and the
        tokens' slots in it, K and V rows go there instead."""
        n = pos.numel()
        Qr = self._bf16(n, self.hq)
        Kr, Vr = cache if cache is not None else (self._bf16(n, self.hkv), self._bf16(n, self.hkv))
        bl.bitlinear_qk_rope(Q, K, V, n, self.hq, self.hkv, self.d, self.q_weight, self.k_weight, self.eps, self.table,
                             pos, Qr, Kr, Vr, slots=slots)
        return Qr, Kr, Vr

    def rotate_bwd(self, Q, K, pos, dQr, dKr):
        """(dQ, dK, dq_weight, dk_weight); the last two None without norms."""
        n, norms = pos.numel(), self.q_weight is not None
        dQ, dK = self._bf16(n, self.hq), self._bf16(n, self.hkv)
        gq = torch.empty(self.d, device=self.device) if norms else None
        gk = torch.empty(self.d, device=self.device) if norms else None
        ws = self._scratch(bl.bitlinear_qk_rope_bwd_workspace_bytes(self.d)) if norms else None
        bl.bitlinear_qk_rope_bwd(Q if norms else None, K if norms else None, n, self.hq, self.hkv, self.d,
                                 self.q_weight, self.k_weight, self.eps, self.table, pos, dQr, dKr, dQ, dK, gq, gk, ws=ws)
        return dQ, dK, gq, gk

    def attend(self, Qr, Kr, Vr, cu_q, cu_k, padded=True):
        """(O, lse) of packed sequences; lse of rows of no sequence is undefined."""
        tq, tk, b = Qr.shape[0], Kr.shape[0], cu_q.numel() - 1
        O, lse = self._bf16(tq, self.hq, padded), torch.empty(self.hq, tq, device=self.device)
        ws = self._scratch(bl.bitlinear_attn_fwd_workspace_bytes(b, tq, tk, self.hq, self.hkv, self.d))
        bl.bitlinear_attn_fwd(Qr, Kr, Vr, cu_q, cu_k, b, self.hq, self.hkv, self.d, self.scale, O, lse, ws=ws)
        return O, lse

    def attend_bwd(self, Qr, Kr, Vr, O, lse, dO, cu_q, cu_k, padded=True):
        """(dQr, dKr, dV) for dO in bfloat16 or float32 (the o BitLinear's dX)."""
        tq, tk, b = Qr.shape[0], Kr.shape[0], cu_q.numel() - 1
        dQ, dK, dV = (self._bf16(n, h, padded) for n, h in ((tq, self.hq), (tk, self.hkv), (tk, self.hkv)))
        ws = self._scratch(bl.bitlinear_attn_bwd_workspace_bytes(b, tq, tk, self.hq, self.hkv, self.d))
        bl.bitlinear_attn_bwd(Qr, Kr, Vr, O, lse, dO, cu_q, cu_k, b, self.hq, self.hkv, self.d, self.scale, dQ, dK, dV,
                              ws=ws)
        return dQ, dK, dV

    def attend_cache(self, Qr, cache, pages, page, lens, tree=None):
        """O of each sequence's newest tokens (lens.numel() * draft rows of Qr)
        over its cache of pages."""
        b = lens.numel()
        if b < 1 or Qr.shape[0] % b:
            raise ValueError(f"{Qr.shape[0]} query rows for {b} sequences")
        draft = Qr.shape[0] // b
        O = self._bf16(b * draft, self.hq)
        ws = self._scratch(bl.bitlinear_attn_cache_workspace_bytes(b, draft, self.hq, self.hkv, self.d))
        bl.bitlinear_attn_cache(Qr, cache[0], cache[1], pages, page, lens, tree, b, draft, self.hq, self.hkv, self.d,
                                self.scale, O, ws=ws)
        return O


def dense_to_sparse(step, switch_step, n, m):
    """N:M pattern of a dense-to-sparse schedule: dense (8:8) before
    switch_step, n:m from it on."""
    return (8, 8) if step < switch_step else (n, m)
