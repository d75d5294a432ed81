"""Tensor-level calls of the norm and rotation of queries and keys: marshalling only.

For a selective scan the queries are C and the keys B: ``feature_major=True``
returns them in the layout ``scan_fwd`` and ``state_update`` take.
"""
from __future__ import annotations

import torch

from . import binding as _b
from ._marshal import io_code, launch, need, ptr, workspace as _workspace


def _shape(t, name, dtype, dev):
    """(batch, seqlen, heads, head_dim) and (batch, token, head) strides of an input
    (batch, L, heads, N), (batch, L, N) of one head, or (batch, N) of one token's one head."""
    if t.dtype is not dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if t.device != dev:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, dev))
    s, st = t.shape, t.stride()
    d = len(s)
    if not 2 <= d <= 4:
        raise ValueError("%s has %d dimensions, expected 2 to 4" % (name, d))
    if st[-1] != 1 and s[-1] > 1 and t.numel():
        raise ValueError("%s must have unit stride in its last dimension" % name)
    if d == 4:
        return s, st[:3]
    if d == 3:
        return (s[0], s[1], 1, s[2]), (st[0], st[1], 0)
    return (s[0], 1, 1, s[1]), (st[0], 0, 0)


def _out_shape(d, shape, feature_major):
    """The output's shape for an input of d dimensions."""
    batch, L, heads, n = shape
    if d == 4:
        return (batch, heads, n, L) if feature_major else shape
    if d == 3:
        return (batch, n, L) if feature_major else (batch, L, n)
    return (batch, n)


def _common(q, k, inv_freq, wq, wk, positions, pos0, interleaved, feature_major):
    ref = q if q is not None else k
    if ref is None:
        raise ValueError("q and k are both None")
    io, dtype, dev = io_code(ref, "q" if q is not None else "k")
    sq, stq = (None, None) if q is None else _shape(q, "q", dtype, dev)
    sk, stk = (None, None) if k is None else _shape(k, "k", dtype, dev)
    batch, L, _, n = sq or sk
    if sq and sk and (sk[0] != batch or sk[1] != L or sk[3] != n or q.dim() != k.dim()):
        raise ValueError("q %s and k %s differ in more than their heads" % (tuple(q.shape), tuple(k.shape)))
    rot = 0
    if inv_freq is not None:
        pairs = inv_freq.shape
        if len(pairs) != 1:
            raise ValueError("inv_freq has %d dimensions, expected 1" % len(pairs))
        need((("inv_freq", inv_freq),), torch.float64, pairs, dev)
        rot = 2 * pairs[0]
    need((("wq", wq), ("wk", wk)), torch.float32, (n,), dev)
    if positions is not None:
        flat = ref.dim() == 2 and positions.dim() == 1
        need((("positions", positions),), torch.int64, (batch,) if flat else (batch, L), dev)
    if not -1 << 63 <= pos0 < 1 << 63:
        raise ValueError("pos0 %r is not a 64-bit integer" % (pos0,))
    flags = (_b.SS_QK_INTERLEAVED if interleaved else 0) | (_b.SS_QK_FEATURE_MAJOR if feature_major else 0)
    head = (batch, L, sq[2] if sq else 0, sk[2] if sk else 0, n, rot, io, flags)
    return dev, dtype, (sq, sk), head, (_b._strides(stq), _b._strides(stk))


def qk_norm_rot(q, k, inv_freq=None, wq=None, wk=None, positions=None, pos0=0, *, eps=1e-6, interleaved=False,
                feature_major=False, q_out=None, k_out=None):
    """RMS norm of each head's queries and keys, times a weight, and their rotation by position, in one pass.

    q: (batch, L, heads, N), (batch, L, N) for one head or (batch, N) for one token of
    one head, float32 or bfloat16, unit stride in the last dimension and any others
    (columns of a projection's rows); k the same with heads of its own; either may be
    None.  wq, wk: (N,) float32 or None.  inv_freq: (R/2,) float64, radians per token of
    each rotated pair (None: no rotation): value j pairs with j + R/2, or 2j with 2j + 1
    when interleaved; values from R on are normed only.  positions: (batch, L) int64
    ((batch,) with (batch, N) inputs), or None for pos0 + t (within 2^53).

    Returns (q, k) contiguous in the inputs' shapes, or with feature_major (N one of 1, 2,
    4, 8, 16) as (batch, heads, N, L) or (batch, N, L): the scan's C and B.
    """
    dev, dtype, sides, head, strides = _common(q, k, inv_freq, wq, wk, positions, pos0, interleaved, feature_major)
    outs = []
    for t, side, given, name in ((q, sides[0], q_out, "q_out"), (k, sides[1], k_out, "k_out")):
        if t is None:
            if given is not None:
                raise ValueError("%s is given without its input" % name)
            outs.append(None)
            continue
        shape = _out_shape(t.dim(), side, feature_major)
        if given is None:
            given = t.new_empty(shape)
        else:
            need(((name, given),), dtype, shape, dev)
        outs.append(given)
    launch(dev, _b.lib.ss_qk_norm_rot, *head, eps, ptr(q), strides[0], ptr(k), strides[1], ptr(wq), ptr(wk),
           ptr(inv_freq), ptr(positions), pos0, ptr(outs[0]), ptr(outs[1]))
    return outs[0], outs[1]


def qk_norm_rot_bwd(q, k, inv_freq, dq_out, dk_out, wq=None, wk=None, positions=None, pos0=0, *, eps=1e-6,
                    interleaved=False, feature_major=False, dq=None, dk=None, need_dw=True, workspace=None):
    """Gradients of ``qk_norm_rot`` for upstream gradients dq_out, dk_out (shaped like its
    outputs, contiguous), given the forward's inputs.

    dq, dk: optional tensors shaped like q and k that receive the gradients, under strides
    of their own (columns of one buffer, side by side or head by head).  Returns a dict: dq, dk in the inputs' dtype and
    shapes; dwq, dwk (N,) float32 (None where there is no input, or need_dw is False).
    """
    dev, dtype, sides, head, strides = _common(q, k, inv_freq, wq, wk, positions, pos0, interleaved, feature_major)
    grads, gst = [], []
    for t, side, up, given, name in ((q, sides[0], dq_out, dq, "dq"), (k, sides[1], dk_out, dk, "dk")):
        if t is None:
            if given is not None or up is not None:
                raise ValueError("%s is given without its input" % (name if given is not None else name + "_out"))
            grads.append(None)
            gst.append(None)
            continue
        if up is None:
            raise ValueError("%s_out is None" % name)
        need(((name + "_out", up),), dtype, _out_shape(t.dim(), side, feature_major), dev)
        if given is None:
            given = t.new_empty(t.shape)
        elif given.shape != t.shape:
            raise ValueError("%s has shape %s, expected %s" % (name, tuple(given.shape), tuple(t.shape)))
        grads.append(given)
        gst.append(_b._strides(_shape(given, name, dtype, dev)[1]))
    batch, L, hq, hk, n = head[:5]
    dw = [torch.empty(n, dtype=torch.float32, device=dev) if need_dw and t is not None else None for t in (q, k)]
    keep, ws, nbytes = _workspace(workspace, _b.ss_qk_norm_rot_bwd_workspace_bytes(batch, L, hq, hk, n), dev)
    launch(dev, _b.lib.ss_qk_norm_rot_bwd, *head, eps, ptr(q), strides[0], ptr(k), strides[1], ptr(wq), ptr(wk),
           ptr(inv_freq), ptr(positions), pos0, ptr(dq_out), ptr(dk_out), ptr(grads[0]), gst[0], ptr(grads[1]), gst[1],
           ptr(dw[0]), ptr(dw[1]), ws, nbytes)
    return dict(dq=grads[0], dk=grads[1], dwq=dw[0], dwk=dw[1])
