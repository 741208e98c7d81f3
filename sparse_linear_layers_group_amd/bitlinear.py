"""Thin Python binding of libbitlinear.so (C ABI in include/bitlinear.h).

Argument marshalling only: each function has the C entry point's name and
argument order, takes torch tensors where the C call takes device pointers,
checks dtype / device / contiguity / size, and passes raw pointers and the
caller's HIP stream (default: torch's current stream).  Every step of the
computation runs in the HIP library; if the library is not built, loading
fails with an error -- there is no fallback path.
"""
import ctypes
import functools
import os
import re

import numpy as np

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("BITLINEAR_LIB") or os.path.join(_HERE, "libbitlinear.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "bitlinear.h")

BL_OK, BL_EINVAL, BL_ESHAPE, BL_EUNSUPPORTED, BL_EWORKSPACE, BL_EHIP = range(6)
BL_GAMMA_DENSE, BL_GAMMA_MASKED = 0, 1


class BitLinearError(RuntimeError):
    def __init__(self, status, where, detail):
        super().__init__(f"{where}: status {status} ({detail})")
        self.status = status


_lib = None
_i64, _int, _sz, _vp = ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p
_f32, _f64 = ctypes.c_float, ctypes.c_double

_SIGS = {
    "bitlinear_packed_bytes": (_sz, [_i64, _i64, _int, _int]),
    "bitlinear_workspace_bytes": (_sz, [_i64, _i64]),
    "bitlinear_fwd_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "bitlinear_bwd_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "bitlinear_quantize_mask": (_int, [_vp, _i64, _i64, _int, _int, _int, _vp, _vp, _vp, _vp, _sz, _vp]),
    "bitlinear_pack": (_int, [_vp, _vp, _vp, _i64, _i64, _int, _int, _vp, _sz, _vp]),
    "bitlinear_fwd": (_int, [_vp, _i64, _i64, _vp, _i64, _int, _int, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "bitlinear_bwd": (_int, [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _int, _int, _vp, _vp, _vp, _sz, _vp]),
    "bitlinear_bwd_tiles": (_int, [_int]),
    "bitlinear_bwd_relu2_gate": (_int, [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _int, _int, _vp, _vp, _vp, _vp,
                                         _vp, _vp, _sz, _vp]),
    "bitlinear_bwd_group_workspace_bytes": (_sz, [_vp, _int, _i64]),
    "bitlinear_bwd_group": (_int, [_vp, _int, _i64, _int, _int, _vp, _sz, _vp]),
    "bitlinear_bwd_group_phase": (_int, [_vp, _int, _i64, _int, _int, _int, _vp, _sz, _vp]),
    "bitlinear_contract_group_workspace_bytes": (_sz, [_vp, _int, _i64, _i64]),
    "bitlinear_contract_group": (_int, [_vp, _int, _vp, _vp, _i64, _i64, _int, _int, _vp, _sz, _vp]),
    "bitlinear_fwd_noalloc": (_int, [_vp, _i64, _i64, _vp, _i64, _int, _int, _vp, _vp, _vp, _vp, _vp, _vp]),
    "bitlinear_sp24_packed_bytes": (_sz, [_i64, _i64]),
    "bitlinear_sp24_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "bitlinear_pack_sp24": (_int, [_vp, _vp, _vp, _i64, _i64, _vp, _sz, _vp]),
    "bitlinear_contract_sp24": (_int, [_vp, _vp, _i64, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _sz, _vp]),
    "bitlinear_act_quant": (_int, [_vp, _i64, _i64, _vp, _vp, _vp]),
    "bitlinear_contract": (_int, [_vp, _vp, _i64, _i64, _vp, _i64, _int, _int, _vp, _vp, _vp, _vp, _sz, _vp]),
    "bitlinear_fwd_bf16": (_int, [_vp, _i64, _i64, _vp, _i64, _int, _int, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "bitlinear_contract_bf16": (_int, [_vp, _vp, _i64, _i64, _vp, _i64, _int, _int, _vp, _vp, _vp, _vp, _sz, _vp]),
    "bitlinear_fwd_group_plan_bytes": (_sz, [_vp, _int, _i64]),
    "bitlinear_fwd_group_plan": (_int, [_vp, _int, _i64, _int, _int, _vp, _sz, _vp]),
    "bitlinear_fwd_group_plan_host": (_int, [_vp, _int, _i64, _int, _int, _vp, _sz]),
    "bitlinear_fwd_group_plan_fuses": (_int, [_vp, _int, _i64, _int, _int]),
    "bitlinear_fwd_group": (_int, [_vp, _int, _int, _int, _vp]),
    "bitlinear_quant_group_workspace_bytes": (_sz, [_vp, _int]),
    "bitlinear_quant_group_plan_bytes": (_sz, [_vp, _int]),
    "bitlinear_quant_group_plan": (_int, [_vp, _int, _int, _int, _int, _vp, _sz, _vp, _sz, _vp]),
    "bitlinear_quant_group": (_int, [_vp, _int, _int, _int, _vp]),
    "bitlinear_latent_update": (_int, [_vp, _vp, _i64, ctypes.c_float, _vp, _vp]),
    "bitlinear_relu2_gate": (_int, [_vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp]),
    "bitlinear_relu2_gate_bwd": (_int, [_vp, _vp, _vp, _i64, _vp, _vp, _vp]),
    "bitlinear_rope_table": (_int, [_i64, _i64, _f64, _vp, _vp]),
    "bitlinear_qk_rope": (_int, [_vp, _vp, _vp, _int] + [_i64] * 7 + [_vp, _vp, _f32, _vp, _i64, _vp, _vp, _i64,
                                                                      _vp, _vp, _vp, _vp]),
    "bitlinear_qk_rope_bwd_workspace_bytes": (_sz, [_i64]),
    "bitlinear_qk_rope_bwd": (_int, [_vp, _vp, _int] + [_i64] * 6 + [_vp, _vp, _f32, _vp, _i64] + [_vp] * 8 +
                              [_sz, _vp]),
    "bitlinear_attn_fwd_workspace_bytes": (_sz, [_i64] * 6),
    "bitlinear_attn_fwd": (_int, [_vp] * 3 + [_i64] * 3 + [_vp] * 2 + [_i64] * 6 + [_f32] + [_vp] * 3 + [_sz, _vp]),
    "bitlinear_attn_bwd_workspace_bytes": (_sz, [_i64] * 6),
    "bitlinear_attn_bwd": (_int, [_vp] * 3 + [_i64] * 3 + [_vp] * 3 + [_int] + [_vp] * 2 + [_i64] * 6 + [_f32] +
                           [_vp] * 4 + [_sz, _vp]),
    "bitlinear_attn_cache_workspace_bytes": (_sz, [_i64] * 5),
    "bitlinear_attn_cache": (_int, [_vp, _i64, _vp, _vp, _i64, _vp, _i64, _i64, _vp, _vp] + [_i64] * 5 + [_f32, _vp, _vp,
                                                                                                   _sz, _vp]),
    "bitlinear_ckpt_pack": (_int, [_vp, _int] + [_i64] * 3 + [_vp] * 3),
    "bitlinear_ckpt_unpack": (_int, [_vp, _vp, _i64, _i64, _vp, _int, _vp]),
    "bitlinear_layernorm": (_int, [_vp, _int] + [_i64] * 3 + [_vp, _vp, _f32, _int, _vp, _int] + [_vp] * 5),
    "bitlinear_layernorm_bwd_workspace_bytes": (_sz, [_i64]),
    "bitlinear_layernorm_bwd": (_int, [_vp, _int, _vp] + [_i64] * 3 + [_vp] * 4 + [_int, _vp, _vp, _int] + [_vp] * 3 +
                                [_sz, _vp]),
    "bitlinear_glu_workspace_bytes": (_sz, [_i64] * 3),
    "bitlinear_glu": (_int, [_vp, _vp, _i64, _i64] + [_vp] * 4 + [_i64, _int, _int, _int, _vp, _int] + [_vp] * 5 +
                      [_sz, _vp]),
    "bitlinear_glu_bwd_workspace_bytes": (_sz, [_i64] * 3),
    "bitlinear_glu_bwd": (_int, [_vp, _int, _int] + [_vp] * 10 + [_i64] * 3 + [_int] * 4 + [_vp] * 4 + [_sz, _vp]),
    "bitlinear_status_string": (ctypes.c_char_p, [_int]),
    "bitlinear_last_error": (ctypes.c_char_p, []),
}


def header_functions():
    """Names of the functions include/bitlinear.h declares."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(bitlinear_\w+)\s*\(", text)))


def lib():
    """Load libbitlinear.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                               "or python -m sparse_linear_layers_group_amd.build")
        h = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(h, name)
            fn.restype = res
            fn.argtypes = args
        _lib = h
    return _lib


# The current stream's handle itself: making a Stream object for it takes 2.5 us
# a call.  (A private name of torch; without it the object is made.)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is None:
            return torch.cuda.current_stream().cuda_stream
        return _raw_stream(torch.cuda.current_device())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


_BF16 = (torch.bfloat16, torch.int16, torch.uint16)


def _ptr(t, dtypes, numel, name, optional=False):
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} has {t.numel()} elements, expected {numel}")
    return t.data_ptr()


def _check(status, where):
    if status != BL_OK:
        detail = lib().bitlinear_last_error().decode() or lib().bitlinear_status_string(status).decode()
        raise BitLinearError(status, where, detail)


def bitlinear_status_string(status):
    return lib().bitlinear_status_string(int(status)).decode()


def bitlinear_last_error():
    return lib().bitlinear_last_error().decode()


def bitlinear_packed_bytes(n_out, k, n, m):
    return int(lib().bitlinear_packed_bytes(int(n_out), int(k), int(n), int(m)))


def bitlinear_workspace_bytes(n_out, k):
    return int(lib().bitlinear_workspace_bytes(int(n_out), int(k)))


def bitlinear_fwd_workspace_bytes(tokens, k, n_out):
    return int(lib().bitlinear_fwd_workspace_bytes(int(tokens), int(k), int(n_out)))


def bitlinear_quantize_mask(W, n_out, k, n, m, gamma_over, mask, wq, gamma, ws, ws_bytes=None,
                            stream=None):
    st = lib().bitlinear_quantize_mask(
        _ptr(W, _BF16, n_out * k, "W"), n_out, k, n, m, gamma_over,
        _ptr(mask, (torch.uint8,), n_out * (k // 8), "mask"),
        _ptr(wq, (torch.int8,), n_out * k, "wq", optional=True),
        _ptr(gamma, (torch.float64,), 1, "gamma"),
        _ptr(ws, (torch.uint8,), None, "ws"),
        ws.numel() if ws_bytes is None else int(ws_bytes), _stream(stream))
    _check(st, "bitlinear_quantize_mask")


def bitlinear_pack(W, mask, gamma, n_out, k, n, m, packed, packed_bytes=None, stream=None):
    st = lib().bitlinear_pack(
        _ptr(W, _BF16, n_out * k, "W"), _ptr(mask, (torch.uint8,), n_out * (k // 8), "mask"),
        _ptr(gamma, (torch.float64,), 1, "gamma"), n_out, k, n, m,
        _ptr(packed, (torch.uint8,), None, "packed"),
        packed.numel() if packed_bytes is None else int(packed_bytes), _stream(stream))
    _check(st, "bitlinear_pack")


def bitlinear_fwd(X, tokens, k, packed, n_out, n, m, gamma, Y, xq, x_scale, acc=None, ws=None,
                  ws_bytes=None, stream=None):
    st = lib().bitlinear_fwd(
        _ptr(X, _BF16, tokens * k, "X"), tokens, k, _ptr(packed, (torch.uint8,), None, "packed"),
        n_out, n, m, _ptr(gamma, (torch.float64,), 1, "gamma"),
        _ptr(Y, (torch.float32,), tokens * n_out, "Y"), _ptr(xq, (torch.int8,), tokens * k, "xq"),
        _ptr(x_scale, (torch.float32,), tokens, "x_scale"),
        _ptr(acc, (torch.int32,), tokens * n_out, "acc", optional=True),
        _ptr(ws, (torch.uint8,), None, "ws", optional=True),
        (ws.numel() if ws is not None else 0) if ws_bytes is None else int(ws_bytes),
        _stream(stream))
    _check(st, "bitlinear_fwd")


def bitlinear_fwd_bf16(X, tokens, k, packed, n_out, n, m, gamma, Y, xq, x_scale, acc=None, ws=None,
                       ws_bytes=None, stream=None):
    """bitlinear_fwd with bf16 Y (a bfloat16 tensor of tokens * n_out)."""
    st = lib().bitlinear_fwd_bf16(
        _ptr(X, _BF16, tokens * k, "X"), tokens, k, _ptr(packed, (torch.uint8,), None, "packed"),
        n_out, n, m, _ptr(gamma, (torch.float64,), 1, "gamma"),
        _ptr(Y, _BF16, tokens * n_out, "Y"), _ptr(xq, (torch.int8,), tokens * k, "xq"),
        _ptr(x_scale, (torch.float32,), tokens, "x_scale"),
        _ptr(acc, (torch.int32,), tokens * n_out, "acc", optional=True),
        _ptr(ws, (torch.uint8,), None, "ws", optional=True),
        (ws.numel() if ws is not None else 0) if ws_bytes is None else int(ws_bytes),
        _stream(stream))
    _check(st, "bitlinear_fwd_bf16")


def bitlinear_fwd_noalloc(X, tokens, k, packed, n_out, n, m, gamma, Y, xq, x_scale, acc=None, stream=None):
    st = lib().bitlinear_fwd_noalloc(
        _ptr(X, _BF16, tokens * k, "X"), tokens, k, _ptr(packed, (torch.uint8,), None, "packed"),
        n_out, n, m, _ptr(gamma, (torch.float64,), 1, "gamma"),
        _ptr(Y, (torch.float32,), tokens * n_out, "Y"), _ptr(xq, (torch.int8,), tokens * k, "xq"),
        _ptr(x_scale, (torch.float32,), tokens, "x_scale"),
        _ptr(acc, (torch.int32,), tokens * n_out, "acc", optional=True), _stream(stream))
    _check(st, "bitlinear_fwd_noalloc")


def bitlinear_sp24_packed_bytes(n_out, k):
    return int(lib().bitlinear_sp24_packed_bytes(int(n_out), int(k)))


def bitlinear_sp24_workspace_bytes(tokens, k, n_out):
    return int(lib().bitlinear_sp24_workspace_bytes(int(tokens), int(k), int(n_out)))


def bitlinear_pack_sp24(W, mask, gamma, n_out, k, packed, packed_bytes=None, stream=None):
    st = lib().bitlinear_pack_sp24(
        _ptr(W, _BF16, n_out * k, "W"), _ptr(mask, (torch.uint8,), n_out * (k // 8), "mask"),
        _ptr(gamma, (torch.float64,), 1, "gamma"), n_out, k, _ptr(packed, (torch.uint8,), None, "packed"),
        packed.numel() if packed_bytes is None else int(packed_bytes), _stream(stream))
    _check(st, "bitlinear_pack_sp24")


def bitlinear_contract_sp24(xq, x_scale, tokens, k, packed, n_out, gamma, Y, acc=None, ws=None, ws_bytes=None,
                            stream=None):
    st = lib().bitlinear_contract_sp24(
        _ptr(xq, (torch.int8,), tokens * k, "xq"), _ptr(x_scale, (torch.float32,), tokens, "x_scale"),
        tokens, k, _ptr(packed, (torch.uint8,), None, "packed"), n_out, _ptr(gamma, (torch.float64,), 1, "gamma"),
        _ptr(Y, (torch.float32,), tokens * n_out, "Y"),
        _ptr(acc, (torch.int32,), tokens * n_out, "acc", optional=True),
        _ptr(ws, (torch.uint8,), None, "ws", optional=True),
        (ws.numel() if ws is not None else 0) if ws_bytes is None else int(ws_bytes), _stream(stream))
    _check(st, "bitlinear_contract_sp24")


def bitlinear_bwd_workspace_bytes(tokens, k, n_out):
    return int(lib().bitlinear_bwd_workspace_bytes(int(tokens), int(k), int(n_out)))


def bitlinear_bwd(dY, xq, x_scale, packed, gamma, tokens, k, n_out, n, m, dX, dW, ws=None,
                  ws_bytes=None, stream=None):
    st = lib().bitlinear_bwd(
        _ptr(dY, _BF16, tokens * n_out, "dY"), _ptr(xq, (torch.int8,), tokens * k, "xq", optional=True),
        _ptr(x_scale, (torch.float32,), tokens, "x_scale", optional=True),
        _ptr(packed, (torch.uint8,), None, "packed", optional=True),
        _ptr(gamma, (torch.float64,), 1, "gamma", optional=True), tokens, k, n_out, n, m,
        _ptr(dX, (torch.float32,), tokens * k, "dX", optional=True),
        _ptr(dW, (torch.float32,), n_out * k, "dW", optional=True),
        _ptr(ws, (torch.uint8,), None, "ws", optional=True),
        (ws.numel() if ws is not None else 0) if ws_bytes is None else int(ws_bytes),
        _stream(stream))
    _check(st, "bitlinear_bwd")


class bitlinear_bwd_item(ctypes.Structure):
    """Mirror of the C struct bitlinear_bwd_item (device pointers as ints)."""
    _fields_ = [("dY", _vp), ("xq", _vp), ("x_scale", _vp), ("packed", _vp), ("gamma", _vp),
                ("dX", _vp), ("dW", _vp), ("k", _i64), ("n_out", _i64)]


def make_bwd_items(entries, tokens):
    """entries: dicts with tensors dY, xq, x_scale, packed, gamma, dX (or None),
    dW (or None) and ints k, n_out."""
    arr = (bitlinear_bwd_item * len(entries))()
    for i, e in enumerate(entries):
        k, n_out = int(e["k"]), int(e["n_out"])
        arr[i] = bitlinear_bwd_item(
            _ptr(e["dY"], _BF16, tokens * n_out, "dY"), _ptr(e.get("xq"), (torch.int8,), tokens * k, "xq", optional=True),
            _ptr(e.get("x_scale"), (torch.float32,), tokens, "x_scale", optional=True),
            _ptr(e.get("packed"), (torch.uint8,), None, "packed", optional=True),
            _ptr(e.get("gamma"), (torch.float64,), 1, "gamma", optional=True),
            _ptr(e.get("dX"), (torch.float32,), tokens * k, "dX", optional=True),
            _ptr(e.get("dW"), (torch.float32,), n_out * k, "dW", optional=True), k, n_out)
    return arr


def bitlinear_bwd_group_workspace_bytes(items, count, tokens):
    return int(lib().bitlinear_bwd_group_workspace_bytes(items, int(count), int(tokens)))


def bitlinear_bwd_group(items, count, tokens, n, m, ws=None, ws_bytes=None, stream=None):
    st = lib().bitlinear_bwd_group(items, int(count), int(tokens), n, m,
                                   _ptr(ws, (torch.uint8,), None, "ws", optional=True),
                                   (ws.numel() if ws is not None else 0) if ws_bytes is None else int(ws_bytes),
                                   _stream(stream))
    _check(st, "bitlinear_bwd_group")


BL_BWD_PREPARE = 1
BL_BWD_FINISH = 2


def bitlinear_bwd_group_phase(items, count, tokens, n, m, phase, ws=None, ws_bytes=None, stream=None):
    """One half of bitlinear_bwd_group: BL_BWD_PREPARE converts the codes and
    x_q into ws, BL_BWD_FINISH converts dY and runs the products."""
    st = lib().bitlinear_bwd_group_phase(items, int(count), int(tokens), n, m, int(phase),
                                         _ptr(ws, (torch.uint8,), None, "ws", optional=True),
                                         (ws.numel() if ws is not None else 0) if ws_bytes is None else int(ws_bytes),
                                         _stream(stream))
    _check(st, "bitlinear_bwd_group_phase")


def bitlinear_bwd_relu2_gate(dY, xq, x_scale, packed, gamma, tokens, k, n_out, n, m, G, U, dG, dU, dW=None,
                             ws=None, ws_bytes=None, stream=None):
    """The down projection's backward with the squared-ReLU gating backward
    fused into its dX epilogue: dG, dU (bfloat16, tokens * k) and dW."""
    st = lib().bitlinear_bwd_relu2_gate(
        _ptr(dY, _BF16, tokens * n_out, "dY"), _ptr(xq, (torch.int8,), tokens * k, "xq", optional=True),
        _ptr(x_scale, (torch.float32,), tokens, "x_scale", optional=True),
        _ptr(packed, (torch.uint8,), None, "packed"), _ptr(gamma, (torch.float64,), 1, "gamma"),
        tokens, k, n_out, n, m, _ptr(G, (torch.float32,), tokens * k, "G"), _ptr(U, (torch.float32,), tokens * k, "U"),
        _ptr(dG, _BF16, tokens * k, "dG"), _ptr(dU, _BF16, tokens * k, "dU"),
        _ptr(dW, (torch.float32,), n_out * k, "dW", optional=True), _ptr(ws, (torch.uint8,), None, "ws", optional=True),
        (ws.numel() if ws is not None else 0) if ws_bytes is None else int(ws_bytes), _stream(stream))
    _check(st, "bitlinear_bwd_relu2_gate")


def bitlinear_bwd_tiles(tiles):
    """Fix the backward products' tiles (0: chosen per launch, 1: 128 x 128,
    2: 256 x 128, 3: 256 x 256)."""
    _check(lib().bitlinear_bwd_tiles(int(tiles)), "bitlinear_bwd_tiles")


def bitlinear_latent_update(W_master, dW, count, lr, W, stream=None):
    st = lib().bitlinear_latent_update(
        _ptr(W_master, (torch.float32,), count, "W_master"), _ptr(dW, (torch.float32,), count, "dW"),
        int(count), float(lr), _ptr(W, _BF16, count, "W"), _stream(stream))
    _check(st, "bitlinear_latent_update")


def bitlinear_relu2_gate(G, U, tokens, n, H, xq, x_scale, stream=None):
    st = lib().bitlinear_relu2_gate(
        _ptr(G, (torch.float32,), tokens * n, "G"), _ptr(U, (torch.float32,), tokens * n, "U"), tokens, n,
        _ptr(H, _BF16, tokens * n, "H", optional=True), _ptr(xq, (torch.int8,), tokens * n, "xq"),
        _ptr(x_scale, (torch.float32,), tokens, "x_scale"), _stream(stream))
    _check(st, "bitlinear_relu2_gate")


def bitlinear_relu2_gate_bwd(dH, G, U, count, dG, dU, stream=None):
    st = lib().bitlinear_relu2_gate_bwd(
        _ptr(dH, (torch.float32,), count, "dH"), _ptr(G, (torch.float32,), count, "G"),
        _ptr(U, (torch.float32,), count, "U"), int(count), _ptr(dG, _BF16, count, "dG"),
        _ptr(dU, _BF16, count, "dU"), _stream(stream))
    _check(st, "bitlinear_relu2_gate_bwd")


def bitlinear_act_quant(X, tokens, k, xq, x_scale, stream=None):
    st = lib().bitlinear_act_quant(_ptr(X, _BF16, tokens * k, "X"), tokens, k,
                                   _ptr(xq, (torch.int8,), tokens * k, "xq"),
                                   _ptr(x_scale, (torch.float32,), tokens, "x_scale"), _stream(stream))
    _check(st, "bitlinear_act_quant")


def bitlinear_contract(xq, x_scale, tokens, k, packed, n_out, n, m, gamma, Y, acc=None, ws=None,
                       ws_bytes=None, stream=None):
    st = lib().bitlinear_contract(
        _ptr(xq, (torch.int8,), tokens * k, "xq"), _ptr(x_scale, (torch.float32,), tokens, "x_scale"),
        tokens, k, _ptr(packed, (torch.uint8,), None, "packed"), n_out, n, m,
        _ptr(gamma, (torch.float64,), 1, "gamma"), _ptr(Y, (torch.float32,), tokens * n_out, "Y"),
        _ptr(acc, (torch.int32,), tokens * n_out, "acc", optional=True),
        _ptr(ws, (torch.uint8,), None, "ws", optional=True),
        (ws.numel() if ws is not None else 0) if ws_bytes is None else int(ws_bytes), _stream(stream))
    _check(st, "bitlinear_contract")


class bitlinear_contract_item(ctypes.Structure):
    """Mirror of the C struct bitlinear_contract_item (device pointers as ints)."""
    _fields_ = [("packed", _vp), ("gamma", _vp), ("Y", _vp), ("Y_bf16", _vp), ("n_out", _i64)]


def make_contract_items(entries, tokens):
    """entries: dicts with tensors packed, gamma, Y (float32) or Y_bf16
    (bfloat16), and int n_out."""
    arr = (bitlinear_contract_item * len(entries))()
    for i, e in enumerate(entries):
        n_out = int(e["n_out"])
        arr[i] = bitlinear_contract_item(
            _ptr(e["packed"], (torch.uint8,), None, "packed"), _ptr(e["gamma"], (torch.float64,), 1, "gamma"),
            _ptr(e.get("Y"), (torch.float32,), tokens * n_out, "Y", optional=True),
            _ptr(e.get("Y_bf16"), _BF16, tokens * n_out, "Y_bf16", optional=True), n_out)
    return arr


def bitlinear_contract_group_workspace_bytes(items, count, tokens, k):
    return int(lib().bitlinear_contract_group_workspace_bytes(items, int(count), int(tokens), int(k)))


def bitlinear_contract_group(items, count, xq, x_scale, tokens, k, n, m, ws=None, ws_bytes=None, stream=None):
    st = lib().bitlinear_contract_group(
        items, int(count), _ptr(xq, (torch.int8,), tokens * k, "xq"),
        _ptr(x_scale, (torch.float32,), tokens, "x_scale"), int(tokens), int(k), n, m,
        _ptr(ws, (torch.uint8,), None, "ws", optional=True),
        (ws.numel() if ws is not None else 0) if ws_bytes is None else int(ws_bytes), _stream(stream))
    _check(st, "bitlinear_contract_group")


def bitlinear_contract_bf16(xq, x_scale, tokens, k, packed, n_out, n, m, gamma, Y, acc=None, ws=None,
                            ws_bytes=None, stream=None):
    """bitlinear_contract with bf16 Y (a bfloat16 tensor of tokens * n_out)."""
    st = lib().bitlinear_contract_bf16(
        _ptr(xq, (torch.int8,), tokens * k, "xq"), _ptr(x_scale, (torch.float32,), tokens, "x_scale"),
        tokens, k, _ptr(packed, (torch.uint8,), None, "packed"), n_out, n, m,
        _ptr(gamma, (torch.float64,), 1, "gamma"), _ptr(Y, _BF16, tokens * n_out, "Y"),
        _ptr(acc, (torch.int32,), tokens * n_out, "acc", optional=True),
        _ptr(ws, (torch.uint8,), None, "ws", optional=True),
        (ws.numel() if ws is not None else 0) if ws_bytes is None else int(ws_bytes), _stream(stream))
    _check(st, "bitlinear_contract_bf16")


class bitlinear_fwd_item(ctypes.Structure):
    """Mirror of the C struct bitlinear_fwd_item (device pointers as ints)."""
    _fields_ = [("X", _vp), ("packed", _vp), ("gamma", _vp), ("Y", _vp), ("xq", _vp),
                ("x_scale", _vp), ("k", _i64), ("n_out", _i64)]


def make_fwd_items(entries, tokens):
    """entries: dicts with tensors X, packed, gamma, Y, xq, x_scale and ints k, n_out."""
    arr = (bitlinear_fwd_item * len(entries))()
    for i, e in enumerate(entries):
        k, n_out = int(e["k"]), int(e["n_out"])
        arr[i] = bitlinear_fwd_item(
            _ptr(e["X"], _BF16, tokens * k, "X"), _ptr(e["packed"], (torch.uint8,), None, "packed"),
            _ptr(e["gamma"], (torch.float64,), 1, "gamma"),
            _ptr(e["Y"], (torch.float32,), tokens * n_out, "Y"), _ptr(e["xq"], (torch.int8,), tokens * k, "xq"),
            _ptr(e["x_scale"], (torch.float32,), tokens, "x_scale"), k, n_out)
    return arr


def bitlinear_fwd_group_plan_bytes(items, count, tokens):
    return int(lib().bitlinear_fwd_group_plan_bytes(items, int(count), int(tokens)))


def bitlinear_fwd_group_plan(items, count, tokens, n, m, plan, plan_bytes=None, stream=None):
    st = lib().bitlinear_fwd_group_plan(items, int(count), int(tokens), n, m,
                                        _ptr(plan, (torch.uint8,), None, "plan"),
                                        plan.numel() if plan_bytes is None else int(plan_bytes),
                                        _stream(stream))
    _check(st, "bitlinear_fwd_group_plan")


def bitlinear_fwd_group_plan_host(items, count, tokens, n, m, image):
    """The plan image into a host numpy uint8 array (no device call)."""
    if not (isinstance(image, np.ndarray) and image.dtype == np.uint8 and image.flags["C_CONTIGUOUS"]):
        raise TypeError("image must be a C-contiguous numpy uint8 array")
    st = lib().bitlinear_fwd_group_plan_host(items, int(count), int(tokens), n, m,
                                             image.ctypes.data_as(ctypes.c_void_p), image.nbytes)
    _check(st, "bitlinear_fwd_group_plan_host")


def bitlinear_fwd_group_plan_fuses(items, count, tokens, n, m):
    """True when the plan for these items can run stage 4 (one launch)."""
    st = lib().bitlinear_fwd_group_plan_fuses(items, int(count), int(tokens), n, m)
    if st < 0:
        _check(-st, "bitlinear_fwd_group_plan_fuses")
    return st == 1


def bitlinear_fwd_group(plan, n, m, stages=3, stream=None):
    st = lib().bitlinear_fwd_group(_ptr(plan, (torch.uint8,), None, "plan"), n, m, int(stages),
                                   _stream(stream))
    _check(st, "bitlinear_fwd_group")


class bitlinear_quant_item(ctypes.Structure):
    """Mirror of the C struct bitlinear_quant_item (device pointers as ints)."""
    _fields_ = [("W", _vp), ("mask", _vp), ("gamma", _vp), ("packed", _vp), ("n_out", _i64), ("k", _i64)]


def make_quant_items(entries, n, m):
    """entries: dicts with tensors W, mask, gamma, packed and ints n_out, k."""
    arr = (bitlinear_quant_item * len(entries))()
    for i, e in enumerate(entries):
        n_out, k = int(e["n_out"]), int(e["k"])
        arr[i] = bitlinear_quant_item(
            _ptr(e["W"], _BF16, n_out * k, "W"), _ptr(e["mask"], (torch.uint8,), n_out * (k // 8), "mask"),
            _ptr(e["gamma"], (torch.float64,), 1, "gamma"),
            _ptr(e["packed"], (torch.uint8,), bitlinear_packed_bytes(n_out, k, n, m), "packed"), n_out, k)
    return arr


def bitlinear_quant_group_workspace_bytes(items, count):
    return int(lib().bitlinear_quant_group_workspace_bytes(items, int(count)))


def bitlinear_quant_group_plan_bytes(items, count):
    return int(lib().bitlinear_quant_group_plan_bytes(items, int(count)))


def bitlinear_quant_group_plan(items, count, n, m, gamma_over, ws, plan, ws_bytes=None, plan_bytes=None,
                               stream=None):
    st = lib().bitlinear_quant_group_plan(
        items, int(count), n, m, gamma_over, _ptr(ws, (torch.uint8,), None, "ws"),
        ws.numel() if ws_bytes is None else int(ws_bytes), _ptr(plan, (torch.uint8,), None, "plan"),
        plan.numel() if plan_bytes is None else int(plan_bytes), _stream(stream))
    _check(st, "bitlinear_quant_group_plan")


def bitlinear_quant_group(plan, n, m, gamma_over, stream=None):
    st = lib().bitlinear_quant_group(_ptr(plan, (torch.uint8,), None, "plan"), n, m, gamma_over,
                                     _stream(stream))
    _check(st, "bitlinear_quant_group")


BL_TYPE_F32, BL_TYPE_BF16 = 0, 1
_F32T, _I32T, _U8T, _FLOATS = (torch.float32,), (torch.int32,), (torch.uint8,), (torch.float32, torch.bfloat16)


# The attention-side calls are short (a few microseconds of GPU work), so
# their checks are one pass per tensor; _refuse names what was wrong.
def _refuse(t, dtypes, numel, name, dev):
    _ptr(t, dtypes, numel, name)
    raise ValueError(f"{name} is on {t.device}, the current device is cuda:{dev}")


def _arg(t, dtypes, numel, name, dev):
    """Pointer of a contiguous tensor on device `dev`."""
    try:
        if t.dtype in dtypes and t.get_device() == dev and t.is_contiguous() and numel in (None, t.numel()):
            return t.data_ptr()
    except AttributeError:  # no tensor
        pass
    _refuse(t, dtypes, numel, name, dev)


def _opt(t, dtypes, numel, name, dev):
    return None if t is None else _arg(t, dtypes, numel, name, dev)


def _rows(t, dtypes, width, name, dev, rows=None):
    """(pointer, row stride in elements, rows) of rows of `width` elements:
    [rows, width] or [rows, heads, d], each row contiguous, the rows any
    distance apart; or a contiguous tensor of any shape."""
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes or t.get_device() != dev:
        _ptr(t, dtypes, None, name)
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{dev}")
    n = t.numel() // width if width > 0 else 0
    if n * width != t.numel() or (rows is not None and n != rows):
        raise ValueError(f"{name} has {t.numel()} elements, expected {'rows' if rows is None else rows} x {width}")
    if n == 0 or t.is_contiguous():
        return t.data_ptr(), width, n
    if t.dim() not in (2, 3) or t.shape[0] != n or t.stride(-1) != 1 or (t.dim() == 3 and t.stride(1) != t.shape[2]):
        raise ValueError(f"{name} must have contiguous rows of {width} elements")
    return t.data_ptr(), t.stride(0) if n > 1 else width, n


def _ws(ws, ws_bytes, dev):
    if ws is None:
        return None, 0 if ws_bytes is None else int(ws_bytes)
    return _arg(ws, _U8T, None, "ws", dev), ws.numel() if ws_bytes is None else int(ws_bytes)


def _type_of(name, first, *others):
    """BL_TYPE_* of tensors that share one of the two input types."""
    kind = getattr(first, "dtype", None)
    if kind not in _FLOATS or any(t is not None and t.dtype != kind for t in others):
        raise TypeError(f"{name} must all be float32 or all bfloat16 tensors")
    return BL_TYPE_F32 if kind == torch.float32 else BL_TYPE_BF16


def _table_rows(table, d, dev):
    p = _arg(table, _F32T, None, "table", dev)
    if d < 1 or table.numel() % d:
        raise ValueError(f"table must hold rows of {d} elements")
    return p, table.numel() // d


def bitlinear_rope_table(max_pos, d, base, table, stream=None):
    """Fill table (float32, max_pos * d/2 * 2) with cos and sin of p * base^(-2i/d)."""
    dev = torch.cuda.current_device()
    st = lib().bitlinear_rope_table(max_pos, d, base, _arg(table, _F32T, max_pos * d, "table", dev), _stream(stream))
    _check(st, "bitlinear_rope_table")


def bitlinear_qk_rope(Q, K, V, tokens, hq, hkv, d, q_weight, k_weight, eps, table, pos, Qr, Kr, Vr, slots=None,
                      stream=None):
    """Head norms (with weights) and rotation of Q and K, V copied: bfloat16
    Qr, Kr, Vr.  Q, K, V: float32 or bfloat16 rows, any row stride; max_pos and
    kv_rows are taken from the sizes of table and Kr."""
    dev = torch.cuda.current_device()
    x_type = _type_of("Q, K and V", Q, K, V)
    q, qs, _ = _rows(Q, _FLOATS, hq * d, "Q", dev, tokens)
    k, ks, _ = _rows(K, _FLOATS, hkv * d, "K", dev, tokens)
    v, vs, _ = _rows(V, _FLOATS, hkv * d, "V", dev, tokens) if V is not None else (None, 0, 0)
    kr = _arg(Kr, _BF16, None, "Kr", dev)
    if min(hkv, d) < 1:
        raise ValueError(f"hkv and d must be positive (got {hkv}, {d})")
    kv_rows = Kr.numel() // (hkv * d)
    if kv_rows * hkv * d != Kr.numel():
        raise ValueError(f"Kr must hold rows of {hkv * d} elements")
    t, max_pos = _table_rows(table, d, dev)
    st = lib().bitlinear_qk_rope(
        q, k, v, x_type, qs, ks, vs, tokens, hq, hkv, d, _opt(q_weight, _F32T, d, "q_weight", dev),
        _opt(k_weight, _F32T, d, "k_weight", dev), eps, t, max_pos, _arg(pos, _I32T, tokens, "pos", dev),
        _opt(slots, (torch.int64,), tokens, "slots", dev), kv_rows, _arg(Qr, _BF16, tokens * hq * d, "Qr", dev), kr,
        _opt(Vr, _BF16, Kr.numel(), "Vr", dev), _stream(stream))
    _check(st, "bitlinear_qk_rope")


def bitlinear_qk_rope_bwd_workspace_bytes(d):
    return int(lib().bitlinear_qk_rope_bwd_workspace_bytes(int(d)))


def bitlinear_qk_rope_bwd(Q, K, tokens, hq, hkv, d, q_weight, k_weight, eps, table, pos, dQr, dKr, dQ, dK,
                          dq_weight=None, dk_weight=None, ws=None, ws_bytes=None, stream=None):
    """Backward of bitlinear_qk_rope for Q and K (which may be None without
    weights): bfloat16 dQ, dK and, with weights, float32 dq_weight, dk_weight."""
    dev = torch.cuda.current_device()
    x_type, q, qs, k, ks = BL_TYPE_F32, None, 0, None, 0
    if q_weight is not None:
        x_type = _type_of("Q and K", Q, K)
        q, qs, _ = _rows(Q, _FLOATS, hq * d, "Q", dev, tokens)
        k, ks, _ = _rows(K, _FLOATS, hkv * d, "K", dev, tokens)
    t, max_pos = _table_rows(table, d, dev)
    w, wn = _ws(ws, ws_bytes, dev)
    st = lib().bitlinear_qk_rope_bwd(
        q, k, x_type, qs, ks, tokens, hq, hkv, d, _opt(q_weight, _F32T, d, "q_weight", dev),
        _opt(k_weight, _F32T, d, "k_weight", dev), eps, t, max_pos, _arg(pos, _I32T, tokens, "pos", dev),
        _arg(dQr, _BF16, tokens * hq * d, "dQr", dev), _arg(dKr, _BF16, tokens * hkv * d, "dKr", dev),
        _arg(dQ, _BF16, tokens * hq * d, "dQ", dev), _arg(dK, _BF16, tokens * hkv * d, "dK", dev),
        _opt(dq_weight, _F32T, d, "dq_weight", dev), _opt(dk_weight, _F32T, d, "dk_weight", dev), w, wn,
        _stream(stream))
    _check(st, "bitlinear_qk_rope_bwd")


def bitlinear_attn_fwd_workspace_bytes(batch, total_q, total_k, hq, hkv, d):
    return int(lib().bitlinear_attn_fwd_workspace_bytes(batch, total_q, total_k, hq, hkv, d))


def bitlinear_attn_fwd(Q, K, V, cu_q, cu_k, batch, hq, hkv, d, scale, O, lse=None, ws=None, ws_bytes=None,
                       stream=None):
    """Causal attention over packed sequences: bfloat16 O, float32 lse
    [hq, total_q].  Q, K, V: bfloat16 rows, any row stride."""
    dev = torch.cuda.current_device()
    q, qs, tq = _rows(Q, _BF16, hq * d, "Q", dev)
    k, ks, tk = _rows(K, _BF16, hkv * d, "K", dev)
    v, vs, _ = _rows(V, _BF16, hkv * d, "V", dev, tk)
    w, wn = _ws(ws, ws_bytes, dev)
    st = lib().bitlinear_attn_fwd(
        q, k, v, qs, ks, vs, _arg(cu_q, _I32T, batch + 1, "cu_q", dev), _arg(cu_k, _I32T, batch + 1, "cu_k", dev),
        batch, tq, tk, hq, hkv, d, scale, _arg(O, _BF16, tq * hq * d, "O", dev), _opt(lse, _F32T, hq * tq, "lse", dev),
        w, wn, _stream(stream))
    _check(st, "bitlinear_attn_fwd")


def bitlinear_attn_bwd_workspace_bytes(batch, total_q, total_k, hq, hkv, d):
    return int(lib().bitlinear_attn_bwd_workspace_bytes(batch, total_q, total_k, hq, hkv, d))


def bitlinear_attn_bwd(Q, K, V, O, lse, dO, cu_q, cu_k, batch, hq, hkv, d, scale, dQ, dK, dV, ws=None, ws_bytes=None,
                       stream=None):
    """Backward of bitlinear_attn_fwd: bfloat16 dQ, dK, dV.  dO: contiguous
    bfloat16 or float32."""
    dev = torch.cuda.current_device()
    q, qs, tq = _rows(Q, _BF16, hq * d, "Q", dev)
    k, ks, tk = _rows(K, _BF16, hkv * d, "K", dev)
    v, vs, _ = _rows(V, _BF16, hkv * d, "V", dev, tk)
    w, wn = _ws(ws, ws_bytes, dev)
    n = tq * hq * d
    st = lib().bitlinear_attn_bwd(
        q, k, v, qs, ks, vs, _arg(O, _BF16, n, "O", dev), _arg(lse, _F32T, hq * tq, "lse", dev),
        _arg(dO, _FLOATS, n, "dO", dev), _type_of("dO", dO), _arg(cu_q, _I32T, batch + 1, "cu_q", dev),
        _arg(cu_k, _I32T, batch + 1, "cu_k", dev), batch, tq, tk, hq, hkv, d, scale, _arg(dQ, _BF16, n, "dQ", dev),
        _arg(dK, _BF16, tk * hkv * d, "dK", dev), _arg(dV, _BF16, tk * hkv * d, "dV", dev), w, wn, _stream(stream))
    _check(st, "bitlinear_attn_bwd")


def bitlinear_attn_cache_workspace_bytes(batch, draft, hq, hkv, d):
    return int(lib().bitlinear_attn_cache_workspace_bytes(batch, draft, hq, hkv, d))


def bitlinear_attn_cache(Q, K, V, pages, page, lens, tree, batch, draft, hq, hkv, d, scale, O, ws=None, ws_bytes=None,
                         stream=None):
    """Attention of batch * draft new tokens over a paged cache: bfloat16 O.
    pages: int32 [batch, max_pages]; tree: int64 or uint64 [batch, draft] bit
    sets, or None (each drafted token sees those before it)."""
    dev = torch.cuda.current_device()
    q, qs, _ = _rows(Q, _BF16, hq * d, "Q", dev, batch * draft)
    k = _arg(K, _BF16, None, "K", dev)
    if min(batch, hkv, d) < 1:
        raise ValueError(f"batch, hkv and d must be positive (got {batch}, {hkv}, {d})")
    rows, width = K.numel() // (hkv * d), pages.numel() // batch
    if rows * hkv * d != K.numel():
        raise ValueError(f"K must hold rows of {hkv * d} elements")
    if width * batch != pages.numel():
        raise ValueError("pages must hold one row per sequence")
    w, wn = _ws(ws, ws_bytes, dev)
    st = lib().bitlinear_attn_cache(
        q, qs, k, _arg(V, _BF16, K.numel(), "V", dev), rows, _arg(pages, _I32T, None, "pages", dev), width, page,
        _arg(lens, _I32T, batch, "lens", dev), _opt(tree, (torch.int64, torch.uint64), batch * draft, "tree", dev),
        batch, draft, hq, hkv, d, scale, _arg(O, _BF16, batch * draft * hq * d, "O", dev), w, wn, _stream(stream))
    _check(st, "bitlinear_attn_cache")


BL_TYPE_Q8 = 2
BL_ACT_RELU2, BL_ACT_SILU = 0, 1
CKPT_BLOCK = 64  # values of a row that share a checkpoint's scale
_I8T, _F64T = (torch.int8,), (torch.float64,)


def _blocks(n):
    return -(-n // CKPT_BLOCK)


_KINDS = {torch.float32: BL_TYPE_F32, torch.bfloat16: BL_TYPE_BF16}


def _stream_on(stream, dev):
    """_stream, for a caller that knows the current device."""
    return _raw_stream(dev) if stream is None and _raw_stream is not None else _stream(stream)


# Sizes that short calls ask for every time: what the C functions answered for the same
# integers (0 for an unsupported layer).
_packed_bytes = functools.lru_cache(maxsize=1024)(bitlinear_packed_bytes)


def _kind(t, name):
    """BL_TYPE_* of one float32 or bfloat16 tensor."""
    kind = _KINDS.get(getattr(t, "dtype", None))
    return _type_of(name, t) if kind is None else kind


def bitlinear_ckpt_pack(X, rows, n, codes, scales, stream=None):
    """8-bit checkpoint of rows of n values: int8 codes [rows, n] and float32
    scales [rows, ceil(n / 64)].  X: float32 or bfloat16 rows, any row stride."""
    dev = torch.cuda.current_device()
    x, xs, _ = _rows(X, _FLOATS, n, "X", dev, rows)
    st = lib().bitlinear_ckpt_pack(
        x, _kind(X, "X"), xs, rows, n, _arg(codes, _I8T, rows * n, "codes", dev),
        _arg(scales, _F32T, rows * _blocks(n), "scales", dev), _stream_on(stream, dev))
    _check(st, "bitlinear_ckpt_pack")


def bitlinear_ckpt_unpack(codes, scales, rows, n, Y, stream=None):
    """The values a checkpoint holds: Y, float32 or bfloat16 [rows, n]."""
    dev = torch.cuda.current_device()
    st = lib().bitlinear_ckpt_unpack(
        _arg(codes, _I8T, rows * n, "codes", dev), _arg(scales, _F32T, rows * _blocks(n), "scales", dev), rows, n,
        _arg(Y, _FLOATS, rows * n, "Y", dev), _kind(Y, "Y"), _stream_on(stream, dev))
    _check(st, "bitlinear_ckpt_unpack")


def bitlinear_layernorm(X, rows, n, weight, bias, eps, center, Y, mean=None, rstd=None, codes=None, scales=None,
                        stream=None):
    """Layer norm of rows (root-mean-square norm with center False): bfloat16
    or float32 Y; mean, rstd (float32 [rows]) and a checkpoint of X where
    given.  X: float32 or bfloat16 rows, any row stride."""
    dev = torch.cuda.current_device()
    x, xs, _ = _rows(X, _FLOATS, n, "X", dev, rows)
    st = lib().bitlinear_layernorm(
        x, _kind(X, "X"), xs, rows, n, _opt(weight, _F32T, n, "weight", dev), _opt(bias, _F32T, n, "bias", dev), eps,
        int(bool(center)), _arg(Y, _FLOATS, rows * n, "Y", dev), _kind(Y, "Y"), _opt(mean, _F32T, rows, "mean", dev),
        _opt(rstd, _F32T, rows, "rstd", dev), _opt(codes, _I8T, rows * n, "codes", dev),
        _opt(scales, _F32T, rows * _blocks(n), "scales", dev), _stream_on(stream, dev))
    _check(st, "bitlinear_layernorm")


def bitlinear_layernorm_bwd_workspace_bytes(n):
    return int(lib().bitlinear_layernorm_bwd_workspace_bytes(int(n)))


def bitlinear_layernorm_bwd(X, x_scales, rows, n, weight, mean, rstd, dY, dX, dweight=None, dbias=None, dR=None, ws=None,
                            ws_bytes=None, stream=None):
    """Backward of bitlinear_layernorm from X (x_scales None) or from the
    checkpoint (X its int8 codes); mean None for a norm that is not centred
    (a tensor, the zeros of an uncentred forward too, makes it a centred one).
    dX: float32 or bfloat16, dR (a residual's gradient, added) of its type."""
    dev = torch.cuda.current_device()
    if getattr(X, "dtype", None) == torch.int8:
        x, xs, x_type = _arg(X, _I8T, rows * n, "X", dev), n, BL_TYPE_Q8
    else:
        x, xs, _ = _rows(X, _FLOATS, n, "X", dev, rows)
        x_type = _kind(X, "X")
    dx_type = _type_of("dX and dR", dX, dR)
    w, wn = _ws(ws, ws_bytes, dev)
    st = lib().bitlinear_layernorm_bwd(
        x, x_type, _opt(x_scales, _F32T, rows * _blocks(n), "x_scales", dev), xs, rows, n,
        _opt(weight, _F32T, n, "weight", dev), _opt(mean, _F32T, rows, "mean", dev), _arg(rstd, _F32T, rows, "rstd", dev),
        _arg(dY, _FLOATS, rows * n, "dY", dev), _kind(dY, "dY"), _opt(dR, _FLOATS, rows * n, "dR", dev),
        _arg(dX, _FLOATS, rows * n, "dX", dev), dx_type, _opt(dweight, _F32T, n, "dweight", dev),
        _opt(dbias, _F32T, n, "dbias", dev), w, wn, _stream_on(stream, dev))
    _check(st, "bitlinear_layernorm_bwd")


def _saved(G, G_scales, U, U_scales, tokens, n_out, dev):
    """(save_type, pointers) of G and U as they are kept: float32, bfloat16 or
    int8 codes with their scales."""
    kind = getattr(G, "dtype", None)
    types = {torch.float32: BL_TYPE_F32, torch.bfloat16: BL_TYPE_BF16, torch.int8: BL_TYPE_Q8}
    if kind not in types or getattr(U, "dtype", None) != kind:
        raise TypeError("G and U must both be float32, bfloat16 or int8 tensors")
    n, ns = tokens * n_out, tokens * _blocks(n_out)
    return (types[kind], _arg(G, (kind,), n, "G", dev), _opt(G_scales, _F32T, ns, "G_scales", dev),
            _arg(U, (kind,), n, "U", dev), _opt(U_scales, _F32T, ns, "U_scales", dev))


@functools.lru_cache(maxsize=1024)
def _glu_ws_bytes(tokens, k, n_out):
    return int(lib().bitlinear_glu_workspace_bytes(tokens, k, n_out))


def bitlinear_glu_workspace_bytes(tokens, k, n_out):
    return _glu_ws_bytes(int(tokens), int(k), int(n_out))


def bitlinear_glu(xq, x_scale, tokens, k, gate, gate_gamma, up, up_gamma, n_out, n, m, act, H, G=None, G_scales=None,
                  U=None, U_scales=None, ws=None, ws_bytes=None, stream=None):
    """bfloat16 H = act(G) * U of two packed layers that read the same
    activations; G and U are kept in the type of the tensors given for them
    (float32, bfloat16, or int8 with float32 scales)."""
    dev = torch.cuda.current_device()
    saved = (BL_TYPE_F32, None, None, None, None)
    if G is not None or U is not None:
        saved = _saved(G, G_scales, U, U_scales, tokens, n_out, dev)
    w, wn = _ws(ws, ws_bytes, dev)
    st = lib().bitlinear_glu(
        _arg(xq, _I8T, tokens * k, "xq", dev), _arg(x_scale, _F32T, tokens, "x_scale", dev), tokens, k,
        _packed(gate, n_out, k, n, m, "gate", dev), _arg(gate_gamma, _F64T, 1, "gate_gamma", dev),
        _packed(up, n_out, k, n, m, "up", dev), _arg(up_gamma, _F64T, 1, "up_gamma", dev), n_out, n, m, act,
        _arg(H, _BF16, tokens * n_out, "H", dev), *saved, w, wn, _stream_on(stream, dev))
    _check(st, "bitlinear_glu")


def _packed(t, n_out, k, n, m, name, dev):
    """Packed codes of an [n_out, k] layer (an unsupported layer is refused by
    the call itself)."""
    return _arg(t, _U8T, _packed_bytes(n_out, k, n, m) or None, name, dev)


def bitlinear_glu_bwd_workspace_bytes(tokens, k, n_out):
    return int(lib().bitlinear_glu_bwd_workspace_bytes(int(tokens), int(k), int(n_out)))


def bitlinear_glu_bwd(dH, G, G_scales, U, U_scales, xq, x_scale, gate, gate_gamma, up, up_gamma, tokens, k, n_out, n, m,
                      act, dX, dW_gate, dW_up, ws=None, ws_bytes=None, stream=None):
    """Backward of bitlinear_glu from G and U as they were kept: dX and the two
    weight gradients, all float32 or all bfloat16 (dX, or both dW, may be
    None).  dH: float32 or bfloat16."""
    dev = torch.cuda.current_device()
    save_type, g, gs, u, us = _saved(G, G_scales, U, U_scales, tokens, n_out, dev)
    grads = [t for t in (dX, dW_gate, dW_up) if t is not None]
    grad_type = _type_of("dX, dW_gate and dW_up", *grads) if grads else BL_TYPE_F32
    w, wn = _ws(ws, ws_bytes, dev)
    st = lib().bitlinear_glu_bwd(
        _arg(dH, _FLOATS, tokens * n_out, "dH", dev), _kind(dH, "dH"), save_type, g, gs, u, us,
        _arg(xq, _I8T, tokens * k, "xq", dev), _arg(x_scale, _F32T, tokens, "x_scale", dev),
        _packed(gate, n_out, k, n, m, "gate", dev), _arg(gate_gamma, _F64T, 1, "gate_gamma", dev),
        _packed(up, n_out, k, n, m, "up", dev), _arg(up_gamma, _F64T, 1, "up_gamma", dev), tokens, k, n_out, n, m, act,
        grad_type, _opt(dX, _FLOATS, tokens * k, "dX", dev), _opt(dW_gate, _FLOATS, n_out * k, "dW_gate", dev),
        _opt(dW_up, _FLOATS, n_out * k, "dW_up", dev), w, wn, _stream_on(stream, dev))
    _check(st, "bitlinear_glu_bwd")
