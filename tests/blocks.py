"""The gated delta rule and the norms before and after a block in 64 bits, token by token and row by row, on the CPU; and the
tolerances that the tests of their kernels share.

Tolerances are relative to the 2-norm of a result.  A product of fp32 values in two fp16 planes is within 2^-21 of the sizes of its
terms, a sum in fp32 much closer; a result passes at most eight such products in a row, and keys of unit length with
beta <= 1 let an error grow (through the inverse of a chunk's triangle, and in differences) to four times its size: 8 x 4 x 2^-21
= 2^-16.  A bf16 result is off by half a step, 2^-8, at most, and where only such results follow one fp16 plane (2^-11) of three
factors is used.
"""
from __future__ import annotations

import torch

F32_REL = 2.0 ** -16
BF16_REL = 2.0 ** -8 + 3 * 2.0 ** -11
#: One rounding of a sum in fp32 over a row, of the hardware's root, reciprocal and exponential, a few of them in a row.
NORM_REL = {torch.float32: 2.0 ** -20, torch.bfloat16: 2.0 ** -8}


def rel(got, want):
    got, want = got.detach().double().cpu(), want.detach().double()
    assert got.shape == want.shape, (got.shape, want.shape)
    n = float(want.norm())
    return float((got - want).norm()) / n if n else float(got.norm())


def close(name, got, want, tol):
    assert bool(torch.isfinite(got).all()), name
    r = rel(got, want)
    assert r <= tol, "%s: off by %.3g of its norm, %.3g allowed" % (name, r, tol)


def tolerance(t):
    return BF16_REL if t.dtype == torch.bfloat16 else F32_REL


def gdr64(q, k, v, g, beta, h0, scale):
    """(o, last state) of (batch, L, heads, n) inputs in float64, differentiable."""
    batch, L, hk, dk = q.shape
    hv, dv = v.shape[2:]
    spread = torch.arange(hv) // (hv // hk)
    h = torch.zeros(batch, hv, dk, dv, dtype=torch.float64) if h0 is None else h0
    out = []
    for t in range(L):
        kt, qt = k[:, t][:, spread], q[:, t][:, spread]
        h = h * torch.exp(g[:, t])[..., None, None] if g is not None else h
        u = beta[:, t][..., None] * (v[:, t] - (h * kt[..., None]).sum(-2))
        h = h + kt[..., None] * u[..., None, :]
        out.append((h * qt[..., None]).sum(-2) * scale)
    return (torch.stack(out, 1) if out else torch.zeros(batch, 0, hv, dv, dtype=torch.float64)), h


def norm64(x, w=None, eps=1e-6):
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return y if w is None else y * w


def silu64(z):
    return z / (1 + torch.exp(-z))


def gated64(x, z, w, first, eps=1e-6):
    if z is None:
        return norm64(x, w, eps)
    return norm64(x * silu64(z), w, eps) if first else norm64(x, w, eps) * silu64(z)


def residual64(x, res, w, w_post, post, scale, alpha, eps=1e-6, rounded=None):
    """(y, r); `rounded`: r as it is kept, for y."""
    m = norm64(x, w_post, eps) if post else x
    r = m * alpha if scale is None else m * alpha * scale
    r = r if res is None else res + r
    kept = r if rounded is None else r + (rounded - r).detach()
    return norm64(kept, w, eps), r


def up(t):
    return None if t is None else t.detach().double().cpu()


def leaves(*ts):
    return [None if t is None else up(t).requires_grad_() for t in ts]
