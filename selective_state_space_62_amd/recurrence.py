"""Tensor-level calls of the gated linear recurrence: marshalling only.

Every call checks dtypes, shapes, devices and contiguity, allocates outputs and
workspaces with torch on the inputs' device, and calls the library on torch's
current stream of that device.
"""
from __future__ import annotations

import torch

from . import binding as _b
from ._marshal import io_code, launch, need, ptr, workspace as _workspace

_KINDS = {"convex": _b.SS_GLR_CONVEX, "normalised": _b.SS_GLR_NORMALISED}
_F32 = torch.float32


def _checked(x, io_tensors, vectors, kind, shape):
    """The checks that all calls share; returns (device, I/O code, kind code)."""
    io, dtype, dev = io_code(x, "x")
    code = _KINDS.get(kind)
    if code is None:
        raise ValueError("kind must be 'convex' or 'normalised', got %r" % (kind,))
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    need(io_tensors, dtype, shape, dev)
    need(vectors, _F32, shape[1:2], dev)
    return dev, io, code


def glr_ckpt_numel(batch, dim, seqlen) -> int:
    """float32 elements of the buffer glr_fwd(ckpt=...) fills for glr_bwd."""
    return _b.ss_glr_ckpt_bytes(batch, dim, seqlen) // 4


def glr_fwd(x, r, i=None, z=None, decay=None, r_bias=None, i_bias=None, h0=None, *, kind="normalised",
            decay_scale=8.0, y=None, h_final=None, return_final_state=True, ckpt=None, workspace=None):
    """Gated linear recurrence over whole sequences: h_t = a_t h_(t-1) + u_t, y_t = h_t silu(z_t).

    With s = sigmoid(r + r_bias) and iota = sigmoid(i + i_bias) (1 without i):
    kind "convex": a = f + (1 - f) s with f = decay in [0, 1] (None: 0), u = (1 - a) iota x;
    kind "normalised": a = exp(-decay_scale softplus(decay) s), u = sqrt(1 - a^2) iota x.

    x, r, i, z: (batch, D, L), all float32 or all bfloat16; decay, r_bias, i_bias: (D,)
    and h0: (batch, D) float32.  ckpt: optional float32 tensor of glr_ckpt_numel(...)
    elements that receives the states glr_bwd starts from.  A padding token has
    r = +inf (convex) or -inf (normalised) and finite x, i and z: it leaves the state alone.
    Returns (y, h_final); h_final (batch, D) is None when return_final_state is False.
    """
    batch, dim, L = x.shape
    shape = x.shape
    dev, io, k = _checked(x, (("r", r), ("i", i), ("z", z), ("y", y)),
                          (("decay", decay), ("r_bias", r_bias), ("i_bias", i_bias)), kind, shape)
    need((("h0", h0), ("h_final", h_final)), _F32, shape[:2], dev)
    if y is None:
        y = torch.empty_like(x)
    if h_final is None and return_final_state:
        h_final = torch.empty_like(h0) if h0 is not None else torch.empty((batch, dim), dtype=_F32, device=dev)
    if ckpt is not None:
        need((("ckpt", ckpt),), _F32, (glr_ckpt_numel(batch, dim, L),), dev)
    keep, ws, nbytes = _workspace(workspace, _b.ss_glr_fwd_workspace_bytes(batch, dim, L), dev)
    launch(dev, _b.lib.ss_glr_fwd, batch, dim, L, io, k, decay_scale, x.data_ptr(), ptr(r), ptr(i), ptr(z), ptr(decay),
           ptr(r_bias), ptr(i_bias), ptr(h0), y.data_ptr(), ptr(h_final), ptr(ckpt), ws, nbytes)
    return y, h_final


def glr_bwd(x, r, dy, i=None, z=None, decay=None, r_bias=None, i_bias=None, h0=None, dh_final=None, *,
            kind="normalised", decay_scale=8.0, ckpt=None, need_ddecay=True, need_dr_bias=True, need_di_bias=True,
            need_dh0=True, workspace=None):
    """Gradients of ``glr_fwd`` for upstream gradients dy (batch, D, L) and dh_final
    (batch, D) float32 (None = 0), given the forward's inputs and optionally the
    states it stored (ckpt).

    Returns a dict: dx, dr, di, dz shaped like x in its dtype (di, dz None without i,
    z); ddecay (of decay itself; None without decay), dr_bias, di_bias (None without
    i): (D,) and dh0 (batch, D) in float32 (None where not requested).
    """
    batch, dim, L = x.shape
    shape = x.shape
    dev, io, k = _checked(x, (("r", r), ("i", i), ("z", z), ("dy", dy)),
                          (("decay", decay), ("r_bias", r_bias), ("i_bias", i_bias)), kind, shape)
    need((("h0", h0), ("dh_final", dh_final)), _F32, shape[:2], dev)
    if ckpt is not None:
        need((("ckpt", ckpt),), _F32, (glr_ckpt_numel(batch, dim, L),), dev)

    def vec(wanted, *shape):
        return torch.empty(shape, dtype=_F32, device=dev) if wanted else None

    out = dict(dx=torch.empty_like(x), dr=torch.empty_like(x), di=None if i is None else torch.empty_like(x),
               dz=None if z is None else torch.empty_like(x), ddecay=vec(need_ddecay and decay is not None, dim),
               dr_bias=vec(need_dr_bias, dim), di_bias=vec(need_di_bias and i is not None, dim),
               dh0=vec(need_dh0, batch, dim))
    keep, ws, nbytes = _workspace(workspace, _b.ss_glr_bwd_workspace_bytes(batch, dim, L), dev)
    launch(dev, _b.lib.ss_glr_bwd, batch, dim, L, io, k, decay_scale, x.data_ptr(), ptr(r), ptr(i), ptr(z), ptr(decay),
           ptr(r_bias), ptr(i_bias), ptr(h0), ptr(dy), ptr(dh_final), ptr(ckpt), ptr(out["dx"]), ptr(out["dr"]),
           ptr(out["di"]), ptr(out["dz"]), ptr(out["ddecay"]), ptr(out["dr_bias"]), ptr(out["di_bias"]), ptr(out["dh0"]),
           ws, nbytes)
    return out


def glr_step(state, x, r, i=None, z=None, decay=None, r_bias=None, i_bias=None, *, kind="normalised",
             decay_scale=8.0, y=None, state_out=None):
    """One token of ``glr_fwd``: ``state`` (batch, D) float32 is updated in place, or the
    new state is written to state_out.  x, r, i, z: (batch, D).  Returns y (batch, D)."""
    batch, dim = x.shape
    shape = x.shape
    dev, io, k = _checked(x, (("r", r), ("i", i), ("z", z), ("y", y)),
                          (("decay", decay), ("r_bias", r_bias), ("i_bias", i_bias)), kind, shape)
    need((("state", state), ("state_out", state_out)), _F32, shape, dev)
    if y is None:
        y = torch.empty_like(x)
    launch(dev, _b.lib.ss_glr_step, batch, dim, io, k, decay_scale, ptr(state),
           ptr(state if state_out is None else state_out), x.data_ptr(), ptr(r), ptr(i), ptr(z), ptr(decay),
           ptr(r_bias), ptr(i_bias), y.data_ptr())
    return y
