"""Tensor-level calls of the gated linear recurrence: marshalling only.

Every call checks dtypes, shapes, devices and contiguity, allocates outputs and
workspaces with torch on the inputs' device, and calls the library on torch's
current stream of that device.
"""
from __future__ import annotations

import torch

from . import binding as _b
from .torch_ops import _IO, _need, _ptr, _stream

_KINDS = {"convex": _b.SS_GLR_CONVEX, "normalised": _b.SS_GLR_NORMALISED}


def _on(dev, fn, *args):
    """Call fn with dev as the current device (its launches go to dev's stream)."""
    if dev.index is None or dev.index == torch.cuda.current_device():
        fn(*args)
    else:
        with torch.cuda.device(dev):
            fn(*args)


def _checked(x, r, i, z, decay, r_bias, i_bias, kind, shape):
    """The checks that all calls share; returns (device, I/O code, kind code)."""
    if x.dtype not in _IO:
        raise TypeError("x must be float32 or bfloat16")
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("inputs must be on a GPU")
    if kind not in _KINDS:
        raise ValueError("kind must be 'convex' or 'normalised', got %r" % (kind,))
    dim = (shape[1],)
    _need(x, "x", x.dtype, shape, dev)
    _need(r, "r", x.dtype, shape, dev)
    _need(i, "i", x.dtype, shape, dev)
    _need(z, "z", x.dtype, shape, dev)
    _need(decay, "decay", torch.float32, dim, dev)
    _need(r_bias, "r_bias", torch.float32, dim, dev)
    _need(i_bias, "i_bias", torch.float32, dim, dev)
    return dev, _IO[x.dtype], _KINDS[kind]


def _workspace(given, nbytes, dev):
    """(address, bytes) of the caller's workspace, or of a new one; nothing where none is needed."""
    if given is None and nbytes:
        given = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    if given is None:
        return None, None, 0
    have = given.numel() * given.element_size()
    if have < nbytes:
        raise ValueError("workspace has %d bytes, %d needed" % (have, nbytes))
    if given.device != dev or not given.is_contiguous():
        raise ValueError("workspace must be contiguous and on %s" % (dev,))
    return given, given.data_ptr(), have


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
    r = +inf (convex) or -inf (normalised) and a finite x: it leaves the state alone.
    Returns (y, h_final); h_final (batch, D) is None when return_final_state is False.
    """
    batch, dim, L = x.shape
    dev, io, k = _checked(x, r, i, z, decay, r_bias, i_bias, kind, (batch, dim, L))
    _need(h0, "h0", torch.float32, (batch, dim), dev)
    if y is None:
        y = torch.empty_like(x)
    else:
        _need(y, "y", x.dtype, (batch, dim, L), dev)
    if h_final is not None:
        _need(h_final, "h_final", torch.float32, (batch, dim), dev)
    elif return_final_state:
        h_final = torch.empty((batch, dim), dtype=torch.float32, device=dev)
    if ckpt is not None:
        _need(ckpt, "ckpt", torch.float32, (glr_ckpt_numel(batch, dim, L),), dev)
    keep, ws, nbytes = _workspace(workspace, _b.ss_glr_fwd_workspace_bytes(batch, dim, L), dev)
    _on(dev, _b.ss_glr_fwd, batch, dim, L, io, k, decay_scale, _ptr(x), _ptr(r), _ptr(i), _ptr(z), _ptr(decay),
        _ptr(r_bias), _ptr(i_bias), _ptr(h0), _ptr(y), _ptr(h_final), _ptr(ckpt), ws, nbytes, _stream(dev))
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
    dev, io, k = _checked(x, r, i, z, decay, r_bias, i_bias, kind, (batch, dim, L))
    _need(dy, "dy", x.dtype, (batch, dim, L), dev)
    _need(h0, "h0", torch.float32, (batch, dim), dev)
    _need(dh_final, "dh_final", torch.float32, (batch, dim), dev)
    if ckpt is not None:
        _need(ckpt, "ckpt", torch.float32, (glr_ckpt_numel(batch, dim, L),), dev)

    def vec(wanted, *shape):
        return torch.empty(shape, dtype=torch.float32, device=dev) if wanted else None

    out = dict(dx=torch.empty_like(x), dr=torch.empty_like(x), di=None if i is None else torch.empty_like(x),
               dz=None if z is None else torch.empty_like(x), ddecay=vec(need_ddecay and decay is not None, dim),
               dr_bias=vec(need_dr_bias, dim), di_bias=vec(need_di_bias and i is not None, dim),
               dh0=vec(need_dh0, batch, dim))
    keep, ws, nbytes = _workspace(workspace, _b.ss_glr_bwd_workspace_bytes(batch, dim, L), dev)
    _on(dev, _b.ss_glr_bwd, batch, dim, L, io, k, decay_scale, _ptr(x), _ptr(r), _ptr(i), _ptr(z), _ptr(decay),
        _ptr(r_bias), _ptr(i_bias), _ptr(h0), _ptr(dy), _ptr(dh_final), _ptr(ckpt), _ptr(out["dx"]), _ptr(out["dr"]),
        _ptr(out["di"]), _ptr(out["dz"]), _ptr(out["ddecay"]), _ptr(out["dr_bias"]), _ptr(out["di_bias"]),
        _ptr(out["dh0"]), ws, nbytes, _stream(dev))
    return out


def glr_step(state, x, r, i=None, z=None, decay=None, r_bias=None, i_bias=None, *, kind="normalised",
             decay_scale=8.0, y=None, state_out=None):
    """One token of ``glr_fwd``: ``state`` (batch, D) float32 is updated in place, or the
    new state is written to state_out.  x, r, i, z: (batch, D).  Returns y (batch, D)."""
    batch, dim = x.shape
    dev, io, k = _checked(x, r, i, z, decay, r_bias, i_bias, kind, (batch, dim))
    _need(state, "state", torch.float32, (batch, dim), dev)
    if state_out is None:
        state_out = state
    else:
        _need(state_out, "state_out", torch.float32, (batch, dim), dev)
    if y is None:
        y = torch.empty_like(x)
    else:
        _need(y, "y", x.dtype, (batch, dim), dev)
    _on(dev, _b.ss_glr_step, batch, dim, io, k, decay_scale, _ptr(state), _ptr(state_out), _ptr(x), _ptr(r), _ptr(i),
        _ptr(z), _ptr(decay), _ptr(r_bias), _ptr(i_bias), _ptr(y), _stream(dev))
    return y
