"""SiLU over the whole range of a gate, both tails, exp's overflow and the
derivative's zero among it: forward in each kernel, backward from G kept in each
type, against binary64."""
import numpy as np
import pytest
import torch

import _ffn_ref as R
from _gpu_ffn import TYPES, activations, dev, empty, host, kept, weight
from sparse_linear_layers_group_amd import bitlinear as bl

pytestmark = pytest.mark.gpu
TINY = 2.0 ** -126  # below it v_rcp_f32 gives 0

# The bounds, in half steps u = 2^-24 of binary32, with e = exp(-g), z = 1 / (1 + e).
# exp(-g) is exp2 of RN(-g log2 e): the product's rounding and the constant's cost 1.5 |g| u of e, v_exp_f32 2 u; so 1 + e
# is off by (1.5 |g| + 2) u e + u (1 + e), relative to 1 + e by at most
#   (1.5 |g| + 2) u min(1, e) + u,
# and v_rcp_f32 adds 2 u: that, with one u to spare, is z's relative error.  Where 1 + e passes 2^126 or is infinite, z may
# be 0 in place of less than 2^-126.
def sigmoid_bound(g):
    with np.errstate(over="ignore"):
        e = np.exp(-g)
    z = 1 / (1 + e)
    return z, ((1.5 * np.abs(g) + 2) * np.minimum(1, e) + 4) * R.U24 * z + TINY


def silu_bounds(g):
    """act, act' and how far each may be off: g z, and z f with f = 1 + g (1 - z), 1 - z rounded once and f once."""
    z, dz = sigmoid_bound(g)
    a = np.abs(g)
    f = 1 + g * (1 - z)
    df = a * (dz + R.U24 * (1 - z)) + R.U24 * np.abs(f) + a * dz * R.U24
    act, slope = g * z, z * f
    return act, a * dz + 2 * R.U24 * np.abs(act), slope, z * df + np.abs(f) * dz + dz * df + 2 * R.U24 * np.abs(slope)


SPECIAL = [-210.0, -150.0, -104.0, -103.9, -103.0, -89.0, -88.73, -88.722, -88.0, -87.4, -87.0, -60.0, -20.0, -17.4, -1.2784645,
           -1e-3, -1e-30, -0.0, 0.0, 1e-30, 1e-3, 1.0, 16.6, 17.4, 60.0, 87.0, 88.73, 100.0, 104.0, 200.0]


def test_the_reference_itself():
    """act' against differences of act in binary64."""
    g = np.linspace(-30, 30, 4001)
    _, _, slope, _ = silu_bounds(g)
    d = 1e-5
    want = (silu_bounds(g + d)[0] - silu_bounds(g - d)[0]) / (2 * d)
    assert np.all(np.abs(slope - want) <= 1e-8 * (1 + np.abs(g)))


# one size for each forward kernel: tokens of their own, tiles that decode for themselves, codes decoded once
@pytest.mark.parametrize("t,k,n_out", [(24, 384, 256), (200, 256, 640), (130, 128, 20608)])
def test_forward(t, k, n_out):
    (gate, cg), (up, cu) = weight(n_out, k, 6, 8, 1), weight(n_out, k, 6, 8, 2)
    xq, xs = activations(t, k, t)
    gg, gu = float(gate.gamma.item()), float(up.gamma.item())
    # every token's largest |G| becomes 220
    top = np.abs(R.project(host(xq), host(xs), cg, gg)).max(1)
    xs.copy_(dev((host(xs) * (220 / top)).astype(np.float32)))
    g, u = R.project(host(xq), host(xs), cg, gg), R.project(host(xq), host(xs), cu, gu)
    for low, high in ((-200, -104), (-104, -88), (-88, -17), (-2, -1), (1, 88), (88, 200)):
        assert ((g > low) & (g < high)).sum() > 20
    act, da, _, _ = silu_bounds(g.astype(np.float64))
    want = act * u
    tol = da * np.abs(u) + (R.UBF + 2 * R.U24) * (np.abs(want) + da * np.abs(u)) + TINY  # bf16's subnormals may go
    for keep in (None, "f32", "bf16", "q8"):
        H, more = empty(t, n_out, dtype=torch.bfloat16), {}
        if keep:
            (G, Gs), (U, Us) = kept(t, n_out, keep), kept(t, n_out, keep)
            more = {"G": G, "G_scales": Gs, "U": U, "U_scales": Us}
        need = bl.bitlinear_glu_workspace_bytes(t, k, n_out)
        bl.bitlinear_glu(xq, xs, t, k, gate.packed, gate.gamma, up.packed, up.gamma, n_out, 6, 8, bl.BL_ACT_SILU, H,
                         ws=torch.empty(need, dtype=torch.uint8, device="cuda") if need else None, **more)
        assert torch.isfinite(H).all()
        assert np.all(np.abs(host(H) - want) <= tol * 1.01)
        if keep == "f32":
            assert np.array_equal(host(G), g) and np.array_equal(host(U), u)


@pytest.mark.parametrize("keep", ["f32", "bf16", "q8"])
@pytest.mark.parametrize("t,k,n_out", [(64, 256, 512), (300, 384, 1152)])
def test_backward(t, k, n_out, keep):
    (gate, cg), (up, cu) = weight(n_out, k, 6, 8, 1), weight(n_out, k, 6, 8, 2)
    xq, xs = activations(t, k, t)
    rng = np.random.default_rng(t)
    g = rng.uniform(-210, 210, size=(t, n_out))
    g[:, ::3] = rng.normal(size=g[:, ::3].shape) * 8
    at = np.arange(t * n_out).reshape(t, n_out)
    g = np.where(at % 5 == 0, np.array(SPECIAL)[at // 5 % len(SPECIAL)], g).astype(np.float32)
    u = rng.normal(size=g.shape).astype(np.float32)
    dh = rng.normal(size=g.shape).astype(np.float32)
    G, U = [], []
    for v, out in ((g, G), (u, U)):
        if keep == "q8":
            c, s = R.ckpt(v)
            out += [torch.from_numpy(c).cuda(), dev(s), R.ckpt_values(c, s)]
        else:
            out += [dev(v, TYPES[keep]), None, v if keep == "f32" else R.bf16(v)]
    g, u = G[2].astype(np.float64), U[2].astype(np.float64)
    assert (np.abs(g) > 100).sum() > 100 and ((g < -87) & (g > -105)).sum() > 100
    outs = [empty(t, k), empty(n_out, k), empty(n_out, k)]
    need = bl.bitlinear_glu_bwd_workspace_bytes(t, k, n_out)
    bl.bitlinear_glu_bwd(dev(dh), G[0], G[1], U[0], U[1], xq, xs, gate.packed, gate.gamma, up.packed, up.gamma, t, k, n_out, 6, 8,
                         bl.BL_ACT_SILU, *outs, ws=torch.empty(need, dtype=torch.uint8, device="cuda"))
    act, da, slope, ds = silu_bounds(g)
    d, gm = dh.astype(np.float64), [float(v.gamma.item()) for v in (gate, up)]
    x, s = host(xq).astype(np.float64), host(xs).astype(np.float64)[:, None]
    c = [v.astype(np.float64) for v in (cg, cu)]
    du, dg = d * act, d * u * slope
    # dh act, dh u slope and the factor behind them: at most three products; then the operand's half step of bf16
    eu, eg = np.abs(d) * da + 4 * R.U24 * np.abs(du), np.abs(d * u) * ds + 4 * R.U24 * np.abs(dg)
    def operand(v, err, factor):
        return (v * factor), (err + R.UBF * (np.abs(v) + err)) * np.abs(factor) + TINY
    og, ou, gs, us = operand(dg, eg, gm[0]), operand(du, eu, gm[1]), operand(dg, eg, s), operand(du, eu, s)
    want = (og[0] @ c[0] + ou[0] @ c[1], gs[0].T @ x, us[0].T @ x)
    err = (og[1] @ np.abs(c[0]) + ou[1] @ np.abs(c[1]), gs[1].T @ np.abs(x), us[1].T @ np.abs(x))
    size = (np.abs(og[0]) @ np.abs(c[0]) + np.abs(ou[0]) @ np.abs(c[1]), np.abs(gs[0]).T @ np.abs(x), np.abs(us[0]).T @ np.abs(x))
    for got, w, e, z, depth in zip(outs, want, err, size, (2 * n_out, t, t)):
        assert torch.isfinite(got).all()
        assert np.all(np.abs(host(got) - w) <= (e + (depth + 8) * R.U24 * (z + e) + R.U24 * np.abs(w)) * 1.01)


def test_gradients_of_single_gates():
    """One token and x_q = 1: dW is s dG and s dU themselves, one bf16 rounding away, at every special gate."""
    n_out, k = 128, 128
    (gate, _), (up, _) = weight(n_out, k, 6, 8, 1), weight(n_out, k, 6, 8, 2)
    g = np.resize(np.array(SPECIAL, np.float32), n_out)[None]
    u, dh = np.full((1, n_out), 1.5, np.float32), np.full((1, n_out), 0.75, np.float32)
    xq, xs = torch.ones(1, k, dtype=torch.int8, device="cuda"), torch.ones(1, device="cuda")
    outs = [empty(1, k), empty(n_out, k), empty(n_out, k)]
    need = bl.bitlinear_glu_bwd_workspace_bytes(1, k, n_out)
    bl.bitlinear_glu_bwd(dev(dh), dev(g), None, dev(u), None, xq, xs, gate.packed, gate.gamma, up.packed, up.gamma, 1, k, n_out,
                         6, 8, bl.BL_ACT_SILU, *outs, ws=torch.empty(need, dtype=torch.uint8, device="cuda"))
    act, da, slope, ds = silu_bounds(g[0].astype(np.float64))
    for got, v, e in ((outs[1], 1.125 * slope, 1.125 * ds), (outs[2], 0.75 * act, 0.75 * da)):
        tol = e + 4 * R.U24 * np.abs(v) + R.UBF * (np.abs(v) + e) + TINY
        assert np.all(np.abs(host(got) - v[:, None]) <= tol[:, None] * 1.01)
