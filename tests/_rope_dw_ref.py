"""The norm weights' gradient in 64 bits with the error its summation allows."""
import torch

F32 = 2.0 ** -24  # half a step of binary32, relative
WAVES = 4 * 768   # wavefronts that share the units of a large call, at most


def weight_gradient(x, dy, cos, sin, eps, heads):
    """(dw, bound) for rows x, dy [tokens, h, d] of one side; heads: those of
    both sides, which a wavefront's unit of 2048 / d head rows is cut from.

    A term is g n with g = R^T dy (two products and a sum: 2 half steps of
    |a c| + |b s|, 3 with the second product's) and n = x / rms (a sum of d
    squares, 16 + log2(d / 16) of them in a row, half of it through the root,
    the root itself 2, and the product: below 16), one more for their product:
    20 half steps.  Sums: a lane adds two terms for each of its wavefront's
    units, one of every WAVES; then 4 joins of lanes at most, 2 of
    wavefronts; binary64 from there, and one rounding."""
    dy, x = dy.double(), x.double()
    t, _, d = dy.shape
    half = d // 2
    a, b = dy[..., :half], dy[..., half:]
    c, s = cos[:, None], sin[:, None]
    g = torch.cat((a * c + b * s, b * c - a * s), -1)
    gabs = torch.cat(((a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()), -1)
    n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    units = t * -(-heads // (2048 // d))
    depth = 2 * -(-units // WAVES) + 4 + 2 + 1
    dw = (g * n).sum((0, 1))
    return dw, F32 * (20 * (gabs * n.abs()).sum((0, 1)) + depth * (g * n).abs().sum((0, 1))) * (1 + 2.0 ** -10)
