"""The gated norm's gradients in one buffer, and weights of every head's own, on the GPU."""
import pytest
import torch

from blocks import NORM_REL, close, gated64, leaves, up
from test_gpu_norms import rn, ss  # noqa: F401

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


@pytest.mark.parametrize("io", [F, BF])
@pytest.mark.parametrize("layout", ["behind", "before", "alternating", "one head"])
def test_gradients_as_columns_of_one_buffer(ss, io, layout):  # noqa: F811
    """dx and dz where x and z stand, columns of a projection's rows: what else is in the rows stays."""
    b, t, h, n = 2, 9, 1 if layout == "one head" else 3, 40
    x, z, dy, w = rn(1, b, t, h, n, io=io), rn(2, b, t, h, n, io=io), rn(3, b, t, h, n, io=io), rn(4, n)
    out = torch.full((b, t, 2 * h * n + 16), 9.0, dtype=io, device="cuda")
    if layout == "alternating":
        both = out[..., 8:8 + 2 * h * n].unflatten(-1, (h, 2, n))
        dx, dz = both[..., 0, :], both[..., 1, :]
    else:
        lo, hi = out[..., 8:8 + h * n].unflatten(-1, (h, n)), out[..., 8 + h * n:8 + 2 * h * n].unflatten(-1, (h, n))
        dx, dz = (hi, lo) if layout == "before" else (lo, hi)
    g = ss.gated_norm_bwd(x, z, dy, w, dx=dx, dz=dz)
    ref = ss.gated_norm_bwd(x, z, dy, w)
    assert torch.equal(g["dx"], ref["dx"]) and torch.equal(g["dz"], ref["dz"]) and torch.equal(g["dw"], ref["dw"])
    assert bool((out[..., :8] == 9).all()) and bool((out[..., 8 + 2 * h * n:] == 9).all())
    with pytest.raises(ss.SsError, match="overlaps dz"):
        ss.gated_norm_bwd(x, z, dy, w, dx=dx, dz=dx)


@pytest.mark.parametrize("tokens,heads,n", [(40_003, 7, 24), (9_001, 40, 128), (3_000, 3, 1000), (2_001, 5, 2048), (70, 300, 8)])
def test_weights_of_every_head_are_all_counted(ss, tokens, heads, n):  # noqa: F811
    """Gradients of every head's weights, of terms that fp32 adds exactly in whatever order: none is lost, none counts for another."""
    x = torch.ones(1, tokens, heads, n, device="cuda")
    dy = torch.randint(-8, 9, (1, tokens, heads, n), generator=torch.Generator().manual_seed(1)).float().cuda()
    g = ss.gated_norm_bwd(x, None, dy, torch.ones(heads, n, device="cuda"), eps=3.0)     # x / sqrt(1 + 3) is 1/2 exactly
    assert torch.equal(g["dw"], dy.double().sum((0, 1)).float() / 2)


def test_more_heads_than_a_launch_has_rows(ss):  # noqa: F811
    """More heads with weights of their own than 2^16."""
    b, t, h, n = 1, 3, 70_001, 8
    x, z, dy, w = rn(1, b, t, h, n), rn(2, b, t, h, n), rn(3, b, t, h, n), rn(4, h, n, scale=0.3, shift=1.0)
    lx, lz, lw = leaves(x, z, w)
    want = gated64(lx, lz, lw, False)
    want.backward(up(dy))
    close("y", ss.gated_norm(x, z, w), want, NORM_REL[F])
    g = ss.gated_norm_bwd(x, z, dy, w)
    close("dz", g["dz"], lz.grad, NORM_REL[F])
    close("dw", g["dw"], lw.grad, 2.0 ** -19)
