"""The bound that the norm weights' gradients are held to (tests/_rope_dw_ref.py)
is one that mistakes do not pass, shown on the CPU: a lost head row and terms
in too few bits."""
import pytest
import torch

import _rope_dw_ref as W


def case(tokens, h, d, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    a = torch.rand(tokens, d // 2, generator=g, dtype=torch.float64) * 6.28
    return n(tokens, h, d).float(), n(tokens, h, d).bfloat16(), a.cos(), a.sin()


def terms(x, dy, c, s, dtype):
    """g n with every operation rounded to dtype."""
    x, dy, c, s = (t.to(dtype) for t in (x, dy, c[:, None], s[:, None]))
    a, b = dy.chunk(2, -1)
    g = torch.cat((a * c + b * s, b * c - a * s), -1)
    return g * (x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6).to(dtype))


@pytest.mark.parametrize("tokens,h,hkv,d", [(5000, 8, 2, 128), (3071, 14, 2, 64), (300, 4, 1, 64)])
def test_mistakes_do_not_pass(tokens, h, hkv, d):
    x, dy, c, s = case(tokens, h, d, tokens)
    dw, err = W.weight_gradient(x, dy, c, s, 1e-6, h + hkv)
    t = terms(x, dy, c, s, torch.float32)
    right = t.double().sum((0, 1))
    assert ((right - dw).abs() <= err).all()
    lanes = t.reshape(-1, d)  # a sum in binary32 for each wavefront, added in binary64
    pad = torch.zeros(-lanes.shape[0] % W.WAVES, d)
    parts = torch.cat((lanes, pad)).view(-1, W.WAVES, d)
    in_lanes = parts[0].clone()
    for p in parts[1:]:
        in_lanes += p
    assert ((in_lanes.double().sum(0) - dw).abs() <= err).all()
    # a head row that is not added
    assert ((right - t[tokens // 2, h // 2].double() - dw).abs() > err).any()
    # terms rounded to bf16
    assert ((t.bfloat16().double().sum((0, 1)) - dw).abs() > err).any()
