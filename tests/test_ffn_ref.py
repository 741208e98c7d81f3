"""The binary64 formulas of the feed-forward side against differences of their
own forwards, and the checkpoint's definition against hand-made blocks."""
import numpy as np
import pytest

import _ffn_ref as R


def directional(f, x, v, h):
    """Central difference of f along v; its error is h^2/6 of the third
    derivative and 2^-53 |f| / h of rounding."""
    return (f(x + h * v) - f(x - h * v)) / (2 * h)


@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("bias", [False, True])
def test_norm_backward_against_differences(center, bias):
    rng = np.random.default_rng(0)
    x, dy = rng.normal(size=(5, 48)) + 0.3, rng.normal(size=(5, 48))
    w, b = rng.normal(size=48), rng.normal(size=48) if bias else None
    _, mean, rstd = R.norm(x, w, b, 1e-5, center)
    dx, dw, db = R.norm_bwd(x, w, mean, rstd, dy, None, center)
    v, u = rng.normal(size=x.shape), rng.normal(size=48)
    loss = lambda x, w, b: (R.norm(x, w, b, 1e-5, center)[0] * dy).sum()  # noqa: E731
    # h = 1e-4: h^2 of third derivatives of a few hundred, 1e-16 * 100 / 1e-4 of rounding
    assert abs(directional(lambda z: loss(z, w, b), x, v, 1e-4) - (dx * v).sum()) < 1e-5
    assert abs(directional(lambda z: loss(x, z, b), w, u, 1e-4) - (dw * u).sum()) < 1e-8
    if bias:
        assert abs(directional(lambda z: loss(x, w, z), b, u, 1e-4) - (db * u).sum()) < 1e-8


@pytest.mark.parametrize("kind", ["relu2", "silu"])
def test_gating_backward_against_differences(kind):
    rng = np.random.default_rng(1)
    t, k, n = 4, 32, 24
    xq = rng.integers(-127, 128, (t, k)).astype(np.float64)
    xs = rng.uniform(0.005, 0.02, t)
    codes = [rng.integers(-1, 2, (n, k)).astype(np.float64) for _ in range(2)]
    gammas, dh = (0.4, 0.7), rng.normal(size=(t, n))

    def loss(x, wg, wu):
        g, u = x @ (gammas[0] * wg).T, x @ (gammas[1] * wu).T
        return (R.act(g, kind)[0] * u * dh).sum()

    x = xq * xs[:, None]
    g, u = x @ (gammas[0] * codes[0]).T, x @ (gammas[1] * codes[1]).T
    (dx, _), (dwg, _), (dwu, _) = R.glu_bwd(dh, g, u, kind, xq, xs, codes, gammas)
    v, w = rng.normal(size=x.shape), rng.normal(size=(n, k))
    # relative to the gradient: h^2 (or h, next to a kink of squared ReLU's slope) of curvature
    for want, f, z in (((dx * v).sum(), lambda y: loss(y, *codes), (x, v)),
                       ((dwg * w).sum() * gammas[0], lambda y: loss(x, y, codes[1]), (codes[0], w)),
                       ((dwu * w).sum() * gammas[1], lambda y: loss(x, codes[0], y), (codes[1], w))):
        got = directional(f, *z, 1e-5)
        assert abs(got - want) <= 1e-4 * (1 + abs(want))


def test_checkpoint_definition():
    x = np.zeros((1, 80), np.float32)
    x[0, :5] = [127, 0.5, 1.5, -0.5, -127]   # a = 127: x inv is x, ties go to even
    x[0, 64:67] = [-3, 1, 2.0 ** -110]       # a short block of its own
    codes, scales = R.ckpt(x)
    assert codes[0, :5].tolist() == [127, 0, 2, 0, -127] and scales[0, 0] == 1
    assert codes[0, 64:67].tolist() == [-127, 42, 0] and scales[0, 1] == np.float32(3) / np.float32(127)
    y = R.ckpt_values(codes, scales)
    # half a step of a / 127, and the roundings of 127 / a, of a / 127 and of the product
    a = np.repeat(np.abs(np.pad(x, ((0, 0), (0, 48))).reshape(1, 2, 64)).max(-1), 64, 1)[:, :80]
    assert np.all(np.abs(y - x) <= a / 254 * (1 + 2.0 ** -14))


def test_checkpoint_edges():
    x = np.zeros((4, 64), np.float32)
    x[0, 3] = np.inf
    x[1, 5], x[1, 6] = np.nan, 3
    x[2, 7] = 2.0 ** -101
    x[3, 8] = 2.0 ** -100
    codes, scales = R.ckpt(x)
    assert np.isnan(R.ckpt_values(codes, scales)[:2]).all()
    assert scales[2, 0] == 0 and not codes[2].any()
    assert codes[3, 8] == 127
