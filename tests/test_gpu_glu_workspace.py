"""The gated feed-forward asks for a workspace where its kernels use one."""
import pytest
import torch

from _gpu_ffn import activations, empty, kept, weight
from sparse_linear_layers_group_amd import bitlinear as bl

pytestmark = pytest.mark.gpu


def test_only_8_bit_values_need_it_at_some_sizes():
    """512 tokens of 8960 outputs: tiles that decode for themselves unless G and U
    are kept in 8 bits, whose tiles are larger."""
    t, k, n_out = 512, 128, 8960
    need = bl.bitlinear_glu_workspace_bytes(t, k, n_out)
    assert need > 0
    (gate, _), (up, _) = weight(n_out, k, 6, 8, 1), weight(n_out, k, 6, 8, 2)
    xq, xs = activations(t, k, 3)

    def run(keep, ws):
        H = empty(t, n_out, dtype=torch.bfloat16)
        more = {}
        if keep:
            (G, Gs), (U, Us) = kept(t, n_out, keep), kept(t, n_out, keep)
            more = {"G": G, "G_scales": Gs, "U": U, "U_scales": Us}
        bl.bitlinear_glu(xq, xs, t, k, gate.packed, gate.gamma, up.packed, up.gamma, n_out, 6, 8, bl.BL_ACT_RELU2, H, ws=ws,
                         **more)
        return [H] + [v for v in more.values() if v is not None]

    for keep in (None, "f32", "bf16"):
        ws = torch.full((need,), 171, dtype=torch.uint8, device="cuda")
        assert all(torch.equal(a, b) for a, b in zip(run(keep, None), run(keep, ws)))
        assert (ws == 171).all()
    with pytest.raises(bl.BitLinearError) as e:
        run("q8", None)
    assert e.value.status == bl.BL_EWORKSPACE
    with pytest.raises(bl.BitLinearError):
        run("q8", torch.empty(need - 256, dtype=torch.uint8, device="cuda"))
    run("q8", torch.empty(need, dtype=torch.uint8, device="cuda"))
