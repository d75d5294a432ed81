"""Tensor-level calls of the norms before and after a block: marshalling only."""
from __future__ import annotations

import torch

from . import binding as _b
from ._marshal import io_code, launch, need, ptr, workspace as _workspace
from .qk import _shape

_F32 = torch.float32


def _gated(x, z, w, eps, gate_first):
    """The checks that both directions share: (device, dtype, the library's first arguments, x's and z's)."""
    io, dtype, dev = io_code(x, "x")
    s, stx = _shape(x, "x", dtype, dev)
    stz = None
    if z is not None:
        if z.shape != x.shape:
            raise ValueError("z has shape %s, expected %s" % (tuple(z.shape), tuple(x.shape)))
        stz = _shape(z, "z", dtype, dev)[1]
    flags = _b.SS_NORM_GATE_FIRST if gate_first else 0
    if w is not None:
        if w.dim() == 2:
            flags |= _b.SS_NORM_HEAD_WEIGHTS
        need((("w", w),), _F32, (s[2], s[3]) if w.dim() == 2 else (s[3],), dev)
    head = (s[0], s[1], s[2], s[3], io, flags, eps)
    return dev, dtype, head, (x.data_ptr(), _b._strides(stx), ptr(z), _b._strides(stz), ptr(w))


def gated_norm(x, z=None, w=None, *, eps=1e-6, gate_first=False, y=None):
    """RMS norm of each row, times a weight, gated by silu(z): w norm(x) silu(z), or w norm(x silu(z)) with gate_first.

    x: (batch, L, heads, N), (batch, L, N) or (batch, N), float32 or bfloat16, N up to 8192,
    unit stride in the last dimension and any others; z: None, or shaped like x under
    strides of its own (columns of a projection's rows).  w: None, (N,) or, a row for every head,
    (heads, N) float32.  Returns y, contiguous in x's shape.
    """
    dev, dtype, head, ins = _gated(x, z, w, eps, gate_first)
    if y is None:
        y = torch.empty(x.shape, dtype=dtype, device=dev)
    else:
        need((("y", y),), dtype, x.shape, dev)
    launch(dev, _b.lib.ss_gated_norm, *head, *ins, y.data_ptr())
    return y


def gated_norm_bwd(x, z, dy, w=None, *, eps=1e-6, gate_first=False, dx=None, dz=None, need_dw=True, workspace=None):
    """Gradients of ``gated_norm`` for the upstream gradient dy (contiguous, shaped like x), given the forward's inputs.

    dx, dz: optional tensors shaped like x that receive the gradients under strides of their
    own, also as columns of the same rows.  Returns a dict: dx, dz (None without z) and dw float32 shaped like w ((N,) without one;
    None where need_dw is False).
    """
    dev, dtype, head, ins = _gated(x, z, w, eps, gate_first)
    if dy is None:
        raise ValueError("dy is None")
    need((("dy", dy),), dtype, x.shape, dev)
    if dz is not None and z is None:
        raise ValueError("dz is given without z")
    grads = []
    for given, name, wanted in ((dx, "dx", True), (dz, "dz", z is not None)):
        if wanted and given is None:
            given = torch.empty(x.shape, dtype=dtype, device=dev)
        elif wanted and given.shape != x.shape:
            raise ValueError("%s has shape %s, expected %s" % (name, tuple(given.shape), tuple(x.shape)))
        grads += [given, _b._strides(_shape(given, name, dtype, dev)[1]) if wanted else None]
    dw = torch.empty(w.shape if w is not None else head[3], dtype=_F32, device=dev) if need_dw else None
    nbytes = _b.ss_gated_norm_bwd_workspace_bytes(*head[:4], head[5]) if need_dw else 0
    keep, ws, nbytes = _workspace(workspace, nbytes, dev)
    launch(dev, _b.lib.ss_gated_norm_bwd, *head, *ins, dy.data_ptr(), grads[0].data_ptr(), grads[1], ptr(grads[2]), grads[3],
           ptr(dw), ws, nbytes)
    return dict(dx=grads[0], dz=grads[2], dw=dw)


def _residual(x, dtype, rdtype, io, vectors, w_post, post, eps, alpha, shape, dev):
    """The library's first arguments for rows of a residual stream."""
    rio = {torch.float32: _b.SS_F32, dtype: io}.get(rdtype)
    if rio is None:
        raise TypeError("the residual has dtype %s, expected torch.float32 or %s" % (rdtype, dtype))
    if len(shape) < 1:
        raise ValueError("x has no dimensions")
    n = shape[-1]
    if w_post is not None and not post:
        raise ValueError("w_post is given without post")
    need(vectors, _F32, (n,), dev)
    rows = 1
    for d in shape[:-1]:
        rows *= d
    return rows, n, io, rio, _b.SS_NORM_POST if post else 0, eps, alpha


def residual_norm(x, res=None, w=None, *, w_post=None, post=False, scale=None, alpha=1.0, eps=1e-6, residual_dtype=None,
                  y=None, res_out=None):
    """A block's output onto the residual stream, and the norm of the sum, in one pass: r = res + alpha scale m,
    y = w norm(r), with m = x, or m = w_post norm(x) with ``post`` (a norm after the block).

    x: (..., N) contiguous, float32 or bfloat16, N up to 8192; res: None (zeros) or shaped like x in
    float32 or x's dtype; scale, w, w_post: (N,) float32 or None.  r has res's dtype (without res:
    residual_dtype, or x's) and is rounded to it before it is normed.  res_out may be res itself.
    Returns (y, r).
    """
    io, dtype, dev = io_code(x, "x")
    shape = x.shape
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    rdtype = res.dtype if res is not None else residual_dtype or dtype
    head = _residual(x, dtype, rdtype, io, (("w", w), ("w_post", w_post), ("scale", scale)), w_post, post, eps, alpha, shape, dev)
    need((("y", y),), dtype, shape, dev)
    need((("res", res), ("res_out", res_out)), rdtype, shape, dev)
    if y is None:
        y = torch.empty_like(x)
    if res_out is None:
        res_out = torch.empty(shape, dtype=rdtype, device=dev)
    launch(dev, _b.lib.ss_residual_norm, *head, x.data_ptr(), ptr(res), ptr(w), ptr(w_post), ptr(scale), y.data_ptr(),
           res_out.data_ptr())
    return y, res_out


def residual_norm_bwd(x, r, dy, dr=None, w=None, *, w_post=None, post=False, scale=None, alpha=1.0, eps=1e-6, dx=None,
                      dres=None, need_dw=True, workspace=None):
    """Gradients of ``residual_norm`` for the upstream gradients dy of y and dr of r (None = 0), given x and the r that
    the forward returned.

    dres may be dr itself.  Returns a dict: dx in x's dtype, dres (of r, and so of res) in r's, and
    float32 dw, dw_post (None without w_post) and dscale (None without scale), None where need_dw is False.
    """
    io, dtype, dev = io_code(x, "x")
    shape = x.shape
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    if r is None or dy is None:
        raise ValueError("%s is None" % ("r" if r is None else "dy"))
    rdtype = r.dtype
    head = _residual(x, dtype, rdtype, io, (("w", w), ("w_post", w_post), ("scale", scale)), w_post, post, eps, alpha, shape, dev)
    need((("dy", dy), ("dx", dx)), dtype, shape, dev)
    need((("r", r), ("dr", dr), ("dres", dres)), rdtype, shape, dev)
    if dx is None:
        dx = torch.empty_like(x)
    if dres is None:
        dres = torch.empty(shape, dtype=rdtype, device=dev)
    n = shape[-1]
    dw, dw_post, dscale = (torch.empty(n, dtype=_F32, device=dev) if need_dw and on else None
                           for on in (True, w_post is not None, scale is not None))
    keep, ws, nbytes = _workspace(workspace, _b.ss_residual_norm_bwd_workspace_bytes(head[0], n) if need_dw else 0, dev)
    launch(dev, _b.lib.ss_residual_norm_bwd, *head, x.data_ptr(), r.data_ptr(), ptr(w), ptr(w_post), ptr(scale), dy.data_ptr(),
           ptr(dr), dx.data_ptr(), dres.data_ptr(), ptr(dw), ptr(dw_post), ptr(dscale), ws, nbytes)
    return dict(dx=dx, dres=dres, dw=dw, dw_post=dw_post, dscale=dscale)
