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
