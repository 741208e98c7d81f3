"""Helpers of the feed-forward side's GPU tests."""
import numpy as np
import torch

from sparse_linear_layers_group_amd import bitlinear as bl
from sparse_linear_layers_group_amd.layer import BitLinearWeight

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "q8": torch.int8}


def dev(x, dtype=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(x)).to("cuda").to(dtype)


def host(t):
    """binary32 (or integer) numpy values of a tensor."""
    return (t.float() if t.is_floating_point() and t.dtype != torch.float64 else t).cpu().numpy()


def empty(*shape, dtype=torch.float32, fill=None):
    t = torch.empty(*shape, dtype=dtype, device="cuda")
    return t if fill is None else t.fill_(fill)


def blocks(n):
    return -(-n // bl.CKPT_BLOCK)


def kept(rows, n, keep):
    return (empty(rows, n, dtype=TYPES[keep]), empty(rows, blocks(n)) if keep == "q8" else None)


def weight(n_out, k, n, m, seed):
    """(layer, int8 codes) of a latent weight drawn from seed."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    W = (torch.randn(n_out, k, generator=gen, device="cuda") * 0.02).bfloat16()
    lw = BitLinearWeight(n_out, k, n, m)
    wq = empty(n_out, k, dtype=torch.int8)
    lw.quantize(W, wq=wq)
    return lw, wq.cpu().numpy()


def activations(t, k, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    X = torch.randn(t, k, generator=gen, device="cuda").bfloat16()
    xq, xs = empty(t, k, dtype=torch.int8), empty(t)
    bl.bitlinear_act_quant(X, t, k, xq, xs)
    return xq, xs
