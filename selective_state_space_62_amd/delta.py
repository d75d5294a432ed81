"""Tensor-level calls of the gated delta rule: marshalling only.

Every call checks dtypes, shapes, devices and strides, allocates outputs and
workspaces with torch on the inputs' device, and calls the library on torch's
current stream of that device.
"""
from __future__ import annotations

import torch

from . import binding as _b
from ._marshal import io_code, launch, need, ptr, workspace as _workspace

_F32 = torch.float32


def _rows(t, name, dims, dtype, dev):
    """The shape of a (batch, L, heads, N) tensor ((batch, heads, N) of one token) and its strides as the library takes them."""
    if t.dtype is not dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if t.device != dev:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, dev))
    s, st = t.shape, t.stride()
    if len(s) != dims:
        raise ValueError("%s has %d dimensions, expected %d" % (name, len(s), dims))
    if st[-1] != 1 and s[-1] > 1 and t.numel():
        raise ValueError("%s must have unit stride in its last dimension" % name)
    return s, _b._strides(st[:3] if dims == 4 else (st[0], 0, st[1]))


def _checked(q, k, v, g, beta, scale, dims):
    """The checks that all calls share: (device, dtype, shape before the heads, the library's first arguments, q's, k's and v's)."""
    io, dtype, dev = io_code(v, "v")
    sq, stq = _rows(q, "q", dims, dtype, dev)
    sk, stk = _rows(k, "k", dims, dtype, dev)
    sv, stv = _rows(v, "v", dims, dtype, dev)
    lead = sv[:-2]
    if sq != sk or sq[:-2] != lead:
        raise ValueError("q %s, k %s and v %s do not fit together" % (tuple(sq), tuple(sk), tuple(sv)))
    hk, dk = sq[-2:]
    hv, dv = sv[-2:]
    if hk < 1 or hv % hk:
        raise ValueError("the %d heads of v are no multiple of the %d heads of q and k" % (hv, hk))
    if beta is None:
        raise ValueError("beta is None")
    need((("g", g), ("beta", beta)), _F32, sv[:-1], dev)
    head = (hk, hv, dk, dv, io, float(dk) ** -0.5 if scale is None else scale)
    return dev, dtype, sv, head, (q.data_ptr(), stq, k.data_ptr(), stk, v.data_ptr(), stv, ptr(g), beta.data_ptr())


def gdr_fwd(q, k, v, g, beta, h0=None, *, scale=None, o=None, h_final=None, return_final_state=True, workspace=None):
    """Gated delta rule over whole sequences, with a (K, V) state S for every value head:

    S' = exp(g_t) S_(t-1);  u = beta_t (v_t - S'^T k_t);  S_t = S' + k_t u^T;  o_t = scale S_t^T q_t.

    q, k: (batch, L, heads_k, K), v: (batch, L, heads_v, V), all float32 or all bfloat16,
    unit stride in the last dimension and any others; heads_v is a multiple of heads_k and
    every key head serves heads_v / heads_k value heads in a row.  g (log decays, None: 0)
    and beta: (batch, L, heads_v), h0: (batch, heads_v, K, V) float32.  K is 1 to 128.
    scale: K^-0.5 unless given.  A padding token has beta = 0, g = 0 and finite q, k and v.
    Returns (o, h_final), o (batch, L, heads_v, V); h_final is None when return_final_state is False.
    """
    dev, dtype, sv, head, ins = _checked(q, k, v, g, beta, scale, 4)
    batch, L, hv, dv = sv
    hk, _, dk = head[:3]
    need((("h0", h0), ("h_final", h_final)), _F32, (batch, hv, dk, dv), dev)
    if o is None:
        o = torch.empty(sv, dtype=dtype, device=dev)
    else:
        need((("o", o),), dtype, sv, dev)
    if h_final is None and return_final_state:
        h_final = torch.empty((batch, hv, dk, dv), dtype=_F32, device=dev)
    keep, ws, nbytes = _workspace(workspace, _b.ss_gdr_fwd_workspace_bytes(batch, L, hk, hv, dk, dv), dev)
    launch(dev, _b.lib.ss_gdr_fwd, batch, L, *head, *ins, ptr(h0), o.data_ptr(), ptr(h_final), ws, nbytes)
    return o, h_final


def gdr_bwd(q, k, v, g, beta, do, h0=None, dh_final=None, *, scale=None, need_dg=True, need_dbeta=True, need_dh0=None,
            workspace=None):
    """Gradients of ``gdr_fwd`` for upstream gradients do (batch, L, heads_v, V), contiguous, and dh_final (batch, heads_v,
    K, V) float32 (None = 0), given the forward's inputs.

    Returns a dict: dq, dk (batch, L, heads_k, K) and dv (batch, L, heads_v, V) in q's dtype, contiguous; dg (None
    without g), dbeta (batch, L, heads_v) and dh0 (batch, heads_v, K, V) float32, None where not needed (dh0: by default
    where h0 is None).
    """
    dev, dtype, sv, head, ins = _checked(q, k, v, g, beta, scale, 4)
    batch, L, hv, dv = sv
    hk, _, dk = head[:3]
    if do is None:
        raise ValueError("do is None")
    need((("do", do),), dtype, sv, dev)
    need((("h0", h0), ("dh_final", dh_final)), _F32, (batch, hv, dk, dv), dev)

    def vec(wanted, *shape):
        return torch.empty(shape, dtype=_F32, device=dev) if wanted else None

    out = dict(dq=torch.empty((batch, L, hk, dk), dtype=dtype, device=dev), dk=torch.empty((batch, L, hk, dk), dtype=dtype, device=dev),
               dv=torch.empty(sv, dtype=dtype, device=dev), dg=vec(need_dg and g is not None, batch, L, hv),
               dbeta=vec(need_dbeta, batch, L, hv), dh0=vec(h0 is not None if need_dh0 is None else need_dh0, batch, hv, dk, dv))
    keep, ws, nbytes = _workspace(workspace, _b.ss_gdr_bwd_workspace_bytes(batch, L, hk, hv, dk, dv), dev)
    launch(dev, _b.lib.ss_gdr_bwd, batch, L, *head, *ins, ptr(h0), do.data_ptr(), ptr(dh_final), ptr(out["dq"]), ptr(out["dk"]),
           ptr(out["dv"]), ptr(out["dg"]), ptr(out["dbeta"]), ptr(out["dh0"]), ws, nbytes)
    return out


def gdr_step(state, q, k, v, g, beta, *, scale=None, o=None, state_out=None):
    """One token of ``gdr_fwd``: ``state`` (batch, heads_v, K, V) float32 is updated in place, or the
    new state is written to state_out.  q, k: (batch, heads_k, K), v: (batch, heads_v, V), g, beta:
    (batch, heads_v).  Returns o (batch, heads_v, V)."""
    dev, dtype, sv, head, ins = _checked(q, k, v, g, beta, scale, 3)
    batch, hv, dv = sv
    if state is None:
        raise ValueError("state is None")
    need((("state", state), ("state_out", state_out)), _F32, (batch, hv, head[2], dv), dev)
    if o is None:
        o = torch.empty(sv, dtype=dtype, device=dev)
    else:
        need((("o", o),), dtype, sv, dev)
    launch(dev, _b.lib.ss_gdr_step, batch, *head, state.data_ptr(),
           (state if state_out is None else state_out).data_ptr(), *ins, o.data_ptr())
    return o
