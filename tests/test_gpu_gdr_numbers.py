"""The gated delta rule's numbers where a norm over all results does not show them: how outputs are rounded, gates and sizes at the
ends of the kernels' ranges, the gates' gradients token by token."""
import math

import pytest
import torch

from blocks import F32_REL, close, gdr64, leaves, rel, up
from test_gpu_gdr import check_bwd, check_fwd, problem, ss, want  # noqa: F401

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32
NAMES = ("q", "k", "v", "g", "beta", "h0")


@pytest.mark.parametrize("size", [(1, 1000, 2, 4, 64, 128), (2, 200, 1, 4, 128, 128), (8, 2048, 2, 16, 64, 64), (1, 90, 1, 3, 30, 50), (4, 16, 2, 2, 64, 64), (3, 600, 1, 2, 128, 200)], ids=str)
def test_bf16_outputs_are_rounded_once(ss, size):  # noqa: F811
    """bf16 outputs are fp32 results rounded once, whatever the length.  An fp32 result off by d, before a rounding to steps of s,
    leaves the 64-bit result's own rounding in a share d / s of the values, each by s: a square of d s in the mean.  With d up to
    2 F32_REL of a value (its own and the mean one's size) and s up to 2^-7 that is 2^-15 2^-7, 2^-11 of the norm."""
    p = problem(*size, BF, seed=2)
    o, _ = ss.gdr_fwd(*[p[n] for n in NAMES])
    wo, _ = want(p)
    assert rel(o, wo.to(BF).double()) <= 2.0 ** -11
