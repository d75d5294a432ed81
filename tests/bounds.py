"""Values with a bound on what fp32 arithmetic may add to them, for tests of fp32 kernels.

A ``V`` holds values in 64 bits and, beside them, how far an fp32 evaluation of the same
formula may be off (first order).  Each operation rounds once: a half step, 2^-24 of its
result.  The hardware's exp2, log2, reciprocal and reciprocal square root are within one
step (two halves) of their result.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24


class V:
    def __init__(self, v, e=0.0):
        self.v = np.asarray(v, dtype=np.float64)
        self.e = np.broadcast_to(np.asarray(e, dtype=np.float64), self.v.shape)

    def __add__(self, o):
        o = o if isinstance(o, V) else V(o)
        v = self.v + o.v
        return V(v, self.e + o.e + U * np.abs(v))

    __radd__ = __add__

    def __neg__(self):
        return V(-self.v, self.e)

    def __sub__(self, o):
        return self + -(o if isinstance(o, V) else V(o))

    def __rsub__(self, o):
        return -self + o

    def __mul__(self, o):
        o = o if isinstance(o, V) else V(o)
        v = self.v * o.v
        return V(v, np.abs(self.v) * o.e + np.abs(o.v) * self.e + U * np.abs(v))

    __rmul__ = __mul__

    def __getitem__(self, at):
        return V(self.v[at], self.e[at])

    def sum(self, axis, adds):
        """A sum in which a value passes `adds` additions at most."""
        return V(self.v.sum(axis), self.e.sum(axis) + adds * U * np.abs(self.v).sum(axis))


def sigmoid(x):
    """1/(1 + exp2(-x log2 e)): the exponent's rounding (twice: product and sum) moves e^-x by that
    much relatively, then exp2, the sum and the reciprocal."""
    s = 0.5 * (1.0 + np.tanh(0.5 * x.v))
    rel = (1.0 - s) * (x.e + 2 * U * np.abs(x.v) + 2 * U) + 3 * U
    return V(s, s * rel)


def silu(z):
    return z * sigmoid(z)


def recur(a, u, h0, adds):
    """h_t = a_t h_(t-1) + u_t along the last axis, a >= 0, token by token: (h, the states before each token).

    The bound holds for every order in which the tokens' maps may be joined: an error made at a
    token reaches t through the decays after it, a relative error of a token's decay through the
    state before it, and each joining rounds a partial result, which is no larger than the same
    recurrence over |u| and |h0|; a token's term passes `adds` such roundings at most."""
    h, mag, err = h0.v.copy(), np.abs(h0.v), h0.e.copy()
    out, bound, before = np.empty_like(a.v), np.empty_like(a.v), np.empty_like(a.v)
    ebefore = np.empty_like(a.v)
    for t in range(a.v.shape[-1]):
        before[..., t], ebefore[..., t] = h, err
        at, ut = a.v[..., t], u.v[..., t]
        err = at * err + a.e[..., t] * mag + u.e[..., t] + 2 * U * (at * mag) + adds * U * np.abs(ut)
        h = at * h + ut
        mag = at * mag + np.abs(ut)
        out[..., t], bound[..., t] = h, err
    return V(out, bound), V(before, ebefore)


def check(name, got, want, half_step, slack=2.0, floor=1e-37):
    """Every value within the bound (twice, for its second order), half a step of its type, and what underflows."""
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == want.v.shape, (name, got.shape, want.v.shape)
    tol = slack * want.e + half_step * np.abs(want.v) * 1.0001 + floor
    off = np.abs(got - want.v)
    bad = ~(off <= tol)
    assert not bad.any(), "%s: %d of %d outside, worst %.3g of its bound at %s (got %r, want %r)" % (
        name, int(bad.sum()), bad.size, float(np.nanmax(off / tol)), np.argwhere(bad)[0].tolist(), got[bad][0], want.v[bad][0])
