"""The gated feed-forward's backward just below its limit, with sums that are
exact: operands are small integers, so every result is known bit for bit."""
import pytest
import torch

from _gpu_ffn import empty, weight
from sparse_linear_layers_group_amd import bitlinear as bl

pytestmark = pytest.mark.gpu


def test_backward_is_exact_at_its_limit():
    """Operands of 2 GiB.  Some tokens of the first, of the last and of a stretch across the middle have a gradient.
    G is 1 or 2, U and the codes -1..1, dH -2..2, both scales 1 and s_t 1: dU = dh g^2 and dG = dh u 2 g are integers up
    to 8, exact in bf16; dX's sums of 2 * 11264 of them stay below 2^18, dW's of 384 of up to 8 * 127 below 2^19."""
    k, n_out = 128, 11264
    tokens = ((1 << 29) // n_out - 1) // 64 * 64 - 3
    gen = torch.Generator(device="cuda").manual_seed(7)
    layers = [weight(n_out, k, 6, 8, i) for i in range(2)]
    gamma = torch.ones(1, dtype=torch.float64, device="cuda")
    def ints(low, high, *shape):
        return torch.randint(low, high + 1, shape, generator=gen, device="cuda")
    rows = torch.cat([torch.arange(128), tokens // 2 - 64 + torch.arange(128), tokens - 128 + torch.arange(128)]).cuda()
    G, U, dH = (torch.zeros(tokens, n_out, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    G[rows] = ints(1, 2, len(rows), n_out).bfloat16()
    U[rows] = ints(-1, 1, len(rows), n_out).bfloat16()
    dH[rows] = ints(-2, 2, len(rows), n_out).bfloat16()
    xq, xs = ints(-127, 127, tokens, k).to(torch.int8), torch.ones(tokens, device="cuda")
    out = [empty(tokens, k, fill=7.0), empty(n_out, k, fill=7.0), empty(n_out, k, fill=7.0)]
    need = bl.bitlinear_glu_bwd_workspace_bytes(tokens, k, n_out)
    assert need > 4 << 30
    bl.bitlinear_glu_bwd(dH, G, None, U, None, xq, xs, layers[0][0].packed, gamma, layers[1][0].packed, gamma, tokens, k, n_out,
                         6, 8, bl.BL_ACT_RELU2, *out, ws=torch.empty(need, dtype=torch.uint8, device="cuda"))
    g, u, dh, x = (v[rows].double() for v in (G, U, dH, xq))
    du, dg = dh * g * g, dh * u * 2 * g
    codes = [torch.from_numpy(c).cuda().double() for _, c in layers]
    assert torch.equal(out[0][rows].double(), dg @ codes[0] + du @ codes[1])
    others = torch.ones(tokens, dtype=torch.bool, device="cuda")
    others[rows] = False
    assert not out[0][others].any()
    assert torch.equal(out[1].double(), dg.t().contiguous() @ x) and torch.equal(out[2].double(), du.t().contiguous() @ x)


@pytest.mark.parametrize("t,k,n_out,dtype", [(547, 896, 4864, torch.float32), (300, 1536, 8960, torch.float32),
                                             (1100, 640, 2560, torch.float32), (33, 256, 4992, torch.float32)])
def test_backward_is_exact_in_every_cut(t, k, n_out, dtype):
    """The same integers where the products are cut along their depth into parts: dX below 2^20, dW's sums of at most
    1100 of up to 8 * 127 below 2^21."""
    gen = torch.Generator(device="cuda").manual_seed(t)
    layers = [weight(n_out, k, 6, 8, i) for i in range(2)]
    gamma = torch.ones(1, dtype=torch.float64, device="cuda")
    def ints(low, high, *shape):
        return torch.randint(low, high + 1, shape, generator=gen, device="cuda")
    G, U, dH = ints(1, 2, t, n_out).bfloat16(), ints(-1, 1, t, n_out).bfloat16(), ints(-2, 2, t, n_out).bfloat16()
    xq, xs = ints(-127, 127, t, k).to(torch.int8), torch.ones(t, device="cuda")
    out = [empty(t, k, dtype=dtype), empty(n_out, k, dtype=dtype), empty(n_out, k, dtype=dtype)]
    need = bl.bitlinear_glu_bwd_workspace_bytes(t, k, n_out)
    bl.bitlinear_glu_bwd(dH, G, None, U, None, xq, xs, layers[0][0].packed, gamma, layers[1][0].packed, gamma, t, k, n_out, 6, 8,
                         bl.BL_ACT_RELU2, *out, ws=torch.empty(need, dtype=torch.uint8, device="cuda"))
    g, u, dh, x = (v.double() for v in (G, U, dH, xq))
    du, dg = dh * g * g, dh * u * 2 * g
    codes = [torch.from_numpy(c).cuda().double() for _, c in layers]
    assert torch.equal(out[0].double(), dg @ codes[0] + du @ codes[1])
    assert torch.equal(out[1].double(), dg.t().contiguous() @ x) and torch.equal(out[2].double(), du.t().contiguous() @ x)
