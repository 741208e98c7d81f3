"""Edges of the backward products' 256-row tiles: odd token counts, rows and
columns that end inside a tile, and memory behind the outputs.  Neighbouring
lanes exchange rows before they store, so an odd last row has a partner that is
out of range.  Every tile size gives the same bits, so the 128 x 128 tiles are
the reference."""
import pytest
import torch

from sparse_linear_layers_group_amd import bitlinear as bl
from sparse_linear_layers_group_amd.layer import BitLinearWeight

pytestmark = pytest.mark.gpu
GUARD = 640


def layer(n_out, k, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    lw = BitLinearWeight(n_out, k, 6, 8)
    lw.quantize((torch.randn(n_out, k, generator=gen, device="cuda") * 0.02).bfloat16())
    return lw


def inputs(tokens, k, n_out, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    xq, xs = torch.empty(tokens, k, dtype=torch.int8, device="cuda"), torch.empty(tokens, device="cuda")
    bl.bitlinear_act_quant(torch.randn(tokens, k, generator=gen, device="cuda").bfloat16(), tokens, k, xq, xs)
    return xq, xs, torch.randn(tokens, n_out, generator=gen, device="cuda").bfloat16(), gen


def guarded(count, dtype=torch.float32):
    return torch.full((count + GUARD,), 5.0, dtype=dtype, device="cuda")


def with_tiles(tiles, call):
    bl.bitlinear_bwd_tiles(tiles)
    try:
        call()
    finally:
        bl.bitlinear_bwd_tiles(0)


SIZES = [(16, 128, 1), (48, 384, 255), (272, 640, 257), (528, 128, 511), (512, 1152, 65), (784, 384, 129)]


@pytest.mark.parametrize("n_out,k,tokens", SIZES)
def test_gradients(n_out, k, tokens):
    lw, (xq, xs, dY, _) = layer(n_out, k, n_out), inputs(tokens, k, n_out, tokens)
    ws = torch.empty(bl.bitlinear_bwd_workspace_bytes(tokens, k, n_out), dtype=torch.uint8, device="cuda")
    out = {}
    for tiles in (1, 2, 3):
        dX, dW = guarded(tokens * k), guarded(n_out * k)
        with_tiles(tiles, lambda: bl.bitlinear_bwd(dY, xq, xs, lw.packed, lw.gamma, tokens, k, n_out, 6, 8,
                                                   dX[:tokens * k], dW[:n_out * k], ws=ws))
        assert (dX[tokens * k:] == 5).all() and (dW[n_out * k:] == 5).all()
        out[tiles] = (dX, dW)
    for tiles in (2, 3):
        assert all(torch.equal(a, b) for a, b in zip(out[tiles], out[1]))


@pytest.mark.parametrize("n_out,k,tokens", SIZES)
def test_gated_gradients(n_out, k, tokens):
    lw, (xq, xs, dY, gen) = layer(n_out, k, n_out), inputs(tokens, k, n_out, tokens)
    count = tokens * k
    G, U = (torch.randn(count, generator=gen, device="cuda") for _ in range(2))
    ws = torch.empty(bl.bitlinear_bwd_workspace_bytes(tokens, k, n_out), dtype=torch.uint8, device="cuda")
    dX, rG, rU = torch.empty(count, device="cuda"), guarded(count, torch.bfloat16), guarded(count, torch.bfloat16)
    with_tiles(1, lambda: bl.bitlinear_bwd(dY, xq, xs, lw.packed, lw.gamma, tokens, k, n_out, 6, 8, dX, None, ws=ws))
    bl.bitlinear_relu2_gate_bwd(dX, G, U, count, rG[:count], rU[:count])
    for tiles in (2, 3):
        dG, dU = guarded(count, torch.bfloat16), guarded(count, torch.bfloat16)
        with_tiles(tiles, lambda: bl.bitlinear_bwd_relu2_gate(dY, xq, xs, lw.packed, lw.gamma, tokens, k, n_out, 6, 8, G, U,
                                                              dG[:count], dU[:count], ws=ws))
        assert torch.equal(dG.view(torch.int16), rG.view(torch.int16))
        assert torch.equal(dU.view(torch.int16), rU.view(torch.int16))
