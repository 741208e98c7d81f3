"""A NaN gate shows in the gated feed-forward, with either activation: a layer's
scale, a token's scale, or one block of an 8-bit checkpoint."""
import pytest
import torch

import _ffn_ref as R
from _gpu_ffn import activations, empty, host, kept, weight
from sparse_linear_layers_group_amd import bitlinear as bl

pytestmark = pytest.mark.gpu
ACT = {"relu2": bl.BL_ACT_RELU2, "silu": bl.BL_ACT_SILU}
NAN = float("nan")
K, N_OUT = 256, 2048
TOKENS = [20, 200, 2900]  # tokens of their own, tiles that decode for themselves, codes decoded once


class Case:
    def __init__(self, t, act, keep):
        self.t, self.act = t, ACT[act]
        self.gate, self.up = (weight(N_OUT, K, 6, 8, i)[0] for i in range(2))
        self.xq, self.xs = activations(t, K, 1)
        self.H, self.G, self.U = empty(t, N_OUT, dtype=torch.bfloat16), kept(t, N_OUT, keep), kept(t, N_OUT, keep)
        self.dH = torch.randn(t, N_OUT, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")

    def scratch(self, need):
        return torch.empty(need, dtype=torch.uint8, device="cuda") if need else None

    def forward(self):
        bl.bitlinear_glu(self.xq, self.xs, self.t, K, self.gate.packed, self.gate.gamma, self.up.packed, self.up.gamma, N_OUT,
                         6, 8, self.act, self.H, G=self.G[0], G_scales=self.G[1], U=self.U[0], U_scales=self.U[1],
                         ws=self.scratch(bl.bitlinear_glu_workspace_bytes(self.t, K, N_OUT)))

    def backward(self):
        """dX, dW_gate, dW_up."""
        out = [empty(self.t, K), empty(N_OUT, K), empty(N_OUT, K)]
        bl.bitlinear_glu_bwd(self.dH, *self.G, *self.U, self.xq, self.xs, self.gate.packed, self.gate.gamma, self.up.packed,
                             self.up.gamma, self.t, K, N_OUT, 6, 8, self.act, *out,
                             ws=self.scratch(bl.bitlinear_glu_bwd_workspace_bytes(self.t, K, N_OUT)))
        return out


@pytest.mark.parametrize("act", ["relu2", "silu"])
@pytest.mark.parametrize("keep", ["f32", "bf16", "q8"])
@pytest.mark.parametrize("t", TOKENS)
def test_a_layers_scale(t, keep, act):
    c = Case(t, act, keep)
    gamma = c.gate.gamma.clone()
    c.gate.gamma.fill_(NAN)
    c.forward()
    dX, dWg, dWu = c.backward()
    assert c.H.isnan().all()
    # (a token whose x_q is 0 at some column adds NaN there as well: dG s_t is NaN)
    assert dX.isnan().all() and dWg.isnan().all() and dWu.isnan().all()
    c.gate.gamma.copy_(gamma)
    c.up.gamma.fill_(NAN)
    c.forward()
    dX, dWg, _ = c.backward()
    assert c.H.isnan().all() and dX.isnan().all() and dWg.isnan().all()


@pytest.mark.parametrize("keep", ["f32", "bf16", "q8"])
@pytest.mark.parametrize("t", TOKENS)
def test_a_tokens_scale_with_squared_relu(t, keep):
    c = Case(t, "relu2", keep)
    c.xs[3] = NAN
    c.forward()
    others = torch.arange(t, device="cuda") != 3
    assert c.H[3].isnan().all() and c.H[others].isfinite().all()
    for v in ((c.G[1], c.U[1]) if keep == "q8" else (c.G[0], c.U[0])):
        assert v[3].isnan().all() and v[others].isfinite().all()


@pytest.mark.parametrize("act", ["relu2", "silu"])
@pytest.mark.parametrize("side", ["G", "U"])
def test_one_block_of_a_checkpoint(side, act):
    t, token, block = 70, 17, 5
    c = Case(t, act, "q8")
    c.forward()
    want = c.backward()
    getattr(c, side)[1][token, block] = NAN
    dX, dWg, dWu = c.backward()
    others = torch.arange(t, device="cuda") != token
    rows = torch.ones(N_OUT, dtype=torch.bool, device="cuda")
    rows[64 * block:64 * block + 64] = False
    assert dX[token].isnan().all() and torch.equal(dX[others], want[0][others])
    assert dWg[~rows].isnan().all() and torch.equal(dWg[rows], want[1][rows])
    # dU = dh act(g) does not read u
    assert torch.equal(dWu, want[2]) if side == "U" else dWu[~rows].isnan().all() and torch.equal(dWu[rows], want[2][rows])


def test_finite_gates_keep_their_bits():
    """Zeros of either sign and the ends of the range."""
    t = 64
    c = Case(t, "relu2", "f32")
    c.forward()
    values = torch.tensor([0.0, -0.0, 1e-45, -1e-45, 1e-20, -3.0, 3.0, 1e19], device="cuda")
    c.G[0].copy_(values.repeat(t * N_OUT // 8).view(t, N_OUT))
    g, u, dh, x, s = (host(v) for v in (c.G[0], c.U[0], c.dH, c.xq, c.xs))
    gm = [float(c.gate.gamma.item()), float(c.up.gamma.item())]
    # 1e19: dU past bf16's operands would be infinite times x_q; keep those outputs out of the sums
    dh = dh.copy()
    dh[:, 7::8] = 0
    c.dH.copy_(torch.from_numpy(dh))
    _, dWg, dWu = c.backward()
    o = [v.astype("f8") for v in R.relu2_operands(dh, g, u, s, gm)]
    for got, op in ((dWg, o[2]), (dWu, o[3])):
        want, size = op.T @ x.astype("f8"), abs(op).T @ abs(x.astype("f8"))
        assert (abs(host(got) - want) <= (t + 8) * R.U24 * size * 1.01 + 1e-30).all()
