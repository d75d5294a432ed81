"""The gated delta rule and the norms before and after a block on the CPU: what their C entry points refuse before they
launch anything, and their size queries.

The addresses are made up and only compared; every call here fails its checks or has nothing to launch.
"""
import pytest

from selective_state_space_62_amd import binding as b

BASE = 0x7F0000000000
GB = 1 << 30
INVALID, UNSUPPORTED, WORKSPACE, OK = b.SS_ERR_INVALID_ARG, b.SS_ERR_UNSUPPORTED, b.SS_ERR_WORKSPACE, b.SS_OK
NAN, INF = float("nan"), float("inf")


def at(k, off=0):
    return BASE + k * GB + off


def gdr(entry="fwd", **kw):
    a = dict(batch=2, seqlen=100, hk=2, hv=4, dk=64, dv=80, io=b.SS_BF16, scale=0.125, q=at(0), qs=(12800, 128, 64), k=at(1),
             ks=(12800, 128, 64), v=at(2), vs=(32000, 320, 80), g=at(3), beta=at(4), h0=at(5), o=at(6), h_final=at(7), ws=at(8),
             ws_bytes=1 << 29, state_in=at(5), state_out=at(5), do=at(10), dh_final=at(11), dq=at(12), dk_=at(13), dv_=at(14), dg=at(15),
             dbeta=at(16), dh0=at(17))
    a.update(kw)
    ins = (a["q"], b._strides(a["qs"]), a["k"], b._strides(a["ks"]), a["v"], b._strides(a["vs"]), a["g"], a["beta"])
    sizes = (a["hk"], a["hv"], a["dk"], a["dv"], a["io"], a["scale"])
    if entry == "fwd":
        st = b.lib.ss_gdr_fwd(a["batch"], a["seqlen"], *sizes, *ins, a["h0"], a["o"], a["h_final"], a["ws"], a["ws_bytes"], None)
    elif entry == "bwd":
        st = b.lib.ss_gdr_bwd(a["batch"], a["seqlen"], *sizes, *ins, a["h0"], a["do"], a["dh_final"], a["dq"], a["dk_"], a["dv_"], a["dg"],
                              a["dbeta"], a["dh0"], a["ws"], a["ws_bytes"], None)
    else:
        st = b.lib.ss_gdr_step(a["batch"], *sizes, a["state_in"], a["state_out"], *ins, a["o"], None)
    return st, b.last_error()


GDR = [
    (dict(io=5), UNSUPPORTED), (dict(batch=0), INVALID), (dict(hk=0), INVALID), (dict(hv=0), INVALID), (dict(hv=3), INVALID),
    (dict(hv=(1 << 20) + 2), INVALID), (dict(dk=0), UNSUPPORTED), (dict(dk=129), UNSUPPORTED), (dict(dv=0), UNSUPPORTED),
    (dict(dv=(1 << 16) + 1), UNSUPPORTED), (dict(batch=(1 << 40) + 1), INVALID), (dict(batch=1 << 40, hv=1 << 18), INVALID),
    (dict(scale=NAN), INVALID), (dict(scale=INF), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(beta=None), INVALID), (dict(q=at(0, 1)), INVALID), (dict(io=b.SS_F32, v=at(2, 2)), INVALID), (dict(g=at(3, 2)), INVALID),
    (dict(beta=at(4, 1)), INVALID), (dict(qs=None), INVALID), (dict(ks=(-1, 128, 64)), INVALID), (dict(vs=(1 << 62, 320, 80)), INVALID),
    (dict(batch=1 << 22, dk=1, dv=1, seqlen=1, qs=(2, 2, 1), ks=(2, 2, 1), vs=(4, 4, 1)), UNSUPPORTED),
]


OUT = [(dict(o=None), INVALID), (dict(o=at(6, 8)), INVALID), (dict(o=at(0)), INVALID), (dict(o=at(4)), INVALID)]


@pytest.mark.parametrize("case,status", GDR + OUT + [
    (dict(seqlen=-1), INVALID), (dict(seqlen=1 << 41), INVALID), (dict(h0=at(5, 2)), INVALID), (dict(h_final=at(7, 2)), INVALID),
    (dict(ws=None), WORKSPACE), (dict(ws=at(8, 128)), WORKSPACE), (dict(ws_bytes=1 << 10), WORKSPACE), (dict(h_final=at(8)), INVALID),
    (dict(h_final=at(5)), INVALID), (dict(h_final=at(6)), INVALID),
])
def test_gdr_fwd_refuses(case, status):
    st, msg = gdr(**case)
    assert st == status and msg, (st, msg)


@pytest.mark.parametrize("case,status", [c for c in GDR if c[0].get("batch") != 1 << 22] + [
    (dict(seqlen=-1), INVALID), (dict(do=None), INVALID), (dict(do=at(10, 8)), INVALID), (dict(dq=None), INVALID), (dict(dk_=None), INVALID),
    (dict(dv_=at(14, 4)), INVALID), (dict(dh_final=at(11, 2)), INVALID), (dict(dg=at(15, 1)), INVALID), (dict(dbeta=at(16, 2)), INVALID),
    (dict(dh0=at(17, 2)), INVALID), (dict(ws=None), WORKSPACE), (dict(ws=at(8, 64)), WORKSPACE), (dict(ws_bytes=1 << 16), WORKSPACE),
    (dict(dq=at(0)), INVALID), (dict(dv_=at(10)), INVALID), (dict(dk_=at(12)), INVALID), (dict(dh0=at(11)), INVALID), (dict(dh0=at(5)), INVALID),
    (dict(dbeta=at(15)), INVALID), (dict(dg=at(8)), INVALID), (dict(vs=(1 << 30, 1 << 22, 80)), UNSUPPORTED), (dict(hv=1 << 10, dv=1 << 12), UNSUPPORTED),
    (dict(batch=1 << 22, dk=1, dv=1, seqlen=1, qs=(2, 2, 1), ks=(2, 2, 1), vs=(4, 4, 1), ws=1 << 40, ws_bytes=1 << 42, h0=None, dh0=None, dh_final=None), UNSUPPORTED),
])
def test_gdr_bwd_refuses(case, status):
    st, msg = gdr("bwd", **case)
    assert st == status and msg, (st, msg)


@pytest.mark.parametrize("case,status", GDR + OUT + [
    (dict(state_in=None), INVALID), (dict(state_out=None), INVALID), (dict(state_out=at(5, 256)), INVALID),
    (dict(state_out=at(9, 2)), INVALID), (dict(state_in=at(5, 2), state_out=at(9)), INVALID), (dict(o=at(5)), INVALID),
    (dict(state_out=at(6)), INVALID), (dict(state_out=at(2)), INVALID),
])
def test_gdr_step_refuses(case, status):
    st, msg = gdr("step", **case)
    assert st == status and msg, (st, msg)


def gated(entry="fwd", **kw):
    a = dict(batch=2, seqlen=10, heads=3, n=40, io=b.SS_BF16, flags=0, eps=1e-6, x=at(0), xs=(1200, 120, 40), z=at(1),
             zs=(2000, 200, 40), w=at(2), y=at(3), dy=at(4), dx=at(5), dxs=(1200, 120, 40), dz=at(6), dzs=(1200, 120, 40),
             dw=at(7), ws=at(8), ws_bytes=1 << 24)
    a.update(kw)
    head = (a["batch"], a["seqlen"], a["heads"], a["n"], a["io"], a["flags"], a["eps"], a["x"], b._strides(a["xs"]), a["z"],
            b._strides(a["zs"]), a["w"])
    if entry == "fwd":
        st = b.lib.ss_gated_norm(*head, a["y"], None)
    else:
        st = b.lib.ss_gated_norm_bwd(*head, a["dy"], a["dx"], b._strides(a["dxs"]), a["dz"], b._strides(a["dzs"]), a["dw"],
                                     a["ws"], a["ws_bytes"], None)
    return st, b.last_error()


GATED = [
    (dict(io=2), UNSUPPORTED), (dict(flags=4), UNSUPPORTED), (dict(eps=0.0), INVALID), (dict(eps=NAN), INVALID), (dict(eps=1e-40), INVALID),
    (dict(batch=0), INVALID), (dict(seqlen=-1), INVALID), (dict(heads=0), INVALID), (dict(heads=(1 << 20) + 1), INVALID),
    (dict(n=0), UNSUPPORTED), (dict(n=8193), UNSUPPORTED), (dict(batch=1 << 16, seqlen=1 << 16, heads=1), UNSUPPORTED),
    (dict(x=None), INVALID), (dict(x=at(0, 1)), INVALID), (dict(xs=None), INVALID), (dict(xs=(0, -1, 0)), INVALID),
    (dict(zs=None), INVALID), (dict(z=at(1, 1)), INVALID), (dict(w=at(2, 2)), INVALID), (dict(zs=(1 << 61, 1, 1)), INVALID),
]


@pytest.mark.parametrize("case,status", GATED + [
    (dict(y=None), INVALID), (dict(y=at(3, 1)), INVALID), (dict(y=at(0)), INVALID), (dict(y=at(1, 16)), INVALID), (dict(y=at(2)), INVALID),
])
def test_gated_norm_refuses(case, status):
    st, msg = gated(**case)
    assert st == status and msg, (st, msg)


@pytest.mark.parametrize("case,status", GATED + [
    (dict(dy=None), INVALID), (dict(dy=at(4, 1)), INVALID), (dict(dx=None), INVALID), (dict(dxs=None), INVALID), (dict(dx=at(5, 1)), INVALID),
    (dict(dz=None), INVALID), (dict(z=None), INVALID), (dict(dzs=None), INVALID), (dict(dw=at(7, 2)), INVALID),
    (dict(dxs=(1200, 120, 39)), INVALID), (dict(dzs=(1200, 100, 40)), INVALID), (dict(dxs=(0, 120, 40)), INVALID),
    (dict(ws=None), WORKSPACE), (dict(ws=at(8, 64)), WORKSPACE), (dict(ws_bytes=16), WORKSPACE), (dict(dx=at(0)), INVALID),
    (dict(dz=at(5)), INVALID), (dict(dw=at(4)), INVALID), (dict(dw=at(8)), INVALID), (dict(dx=at(4)), INVALID),
])
def test_gated_norm_bwd_refuses(case, status):
    st, msg = gated("bwd", **case)
    assert st == status and msg, (st, msg)


def residual(entry="fwd", **kw):
    a = dict(rows=10, n=96, io=b.SS_BF16, rio=b.SS_F32, flags=b.SS_NORM_POST, eps=1e-6, alpha=0.5, x=at(0), res=at(1), w=at(2), w_post=at(3),
             scale=at(4), y=at(5), res_out=at(1), dy=at(6), dres_out=at(7), dx=at(8), dres=at(7), dw=at(9), dw_post=at(10), dscale=at(11),
             ws=at(12), ws_bytes=1 << 24)
    a.update(kw)
    head = [a[k] for k in ("rows", "n", "io", "rio", "flags", "eps", "alpha", "x", "res", "w", "w_post", "scale")]
    if entry == "fwd":
        st = b.lib.ss_residual_norm(*head, a["y"], a["res_out"], None)
    else:
        st = b.lib.ss_residual_norm_bwd(*head, *[a[k] for k in ("dy", "dres_out", "dx", "dres", "dw", "dw_post", "dscale", "ws", "ws_bytes")], None)
    return st, b.last_error()


RESIDUAL = [
    (dict(io=2), UNSUPPORTED), (dict(rio=2), UNSUPPORTED), (dict(io=b.SS_F32, rio=b.SS_BF16), UNSUPPORTED), (dict(flags=8), UNSUPPORTED),
    (dict(flags=1), UNSUPPORTED), (dict(flags=0), INVALID), (dict(eps=-1.0), INVALID), (dict(alpha=NAN), INVALID), (dict(alpha=INF), INVALID), (dict(rows=-1), INVALID),
    (dict(rows=1 << 32), UNSUPPORTED), (dict(n=0), UNSUPPORTED), (dict(n=8193), UNSUPPORTED), (dict(x=None), INVALID), (dict(x=at(0, 1)), INVALID),
    (dict(res=at(1, 2)), INVALID), (dict(w=at(2, 2)), INVALID), (dict(w_post=at(3, 1)), INVALID), (dict(scale=at(4, 2)), INVALID),
]


@pytest.mark.parametrize("case,status", RESIDUAL + [
    (dict(y=None), INVALID), (dict(y=at(5, 1)), INVALID), (dict(y=at(0)), INVALID), (dict(y=at(1)), INVALID), (dict(res_out=at(1, 4)), INVALID),
    (dict(res_out=at(0)), INVALID), (dict(res_out=at(5)), INVALID), (dict(res_out=at(13, 2)), INVALID), (dict(res_out=at(2)), INVALID),
])
def test_residual_norm_refuses(case, status):
    st, msg = residual(**case)
    assert st == status and msg, (st, msg)


@pytest.mark.parametrize("case,status", RESIDUAL + [
    (dict(res=None), INVALID), (dict(dy=None), INVALID), (dict(dx=at(8, 1)), INVALID), (dict(dres=at(13, 2)), INVALID), (dict(dw=at(9, 2)), INVALID),
    (dict(flags=0, w_post=None), INVALID), (dict(flags=0, w_post=None, dw_post=None, x=None), INVALID),
    (dict(ws=None), WORKSPACE), (dict(ws=at(12, 8)), WORKSPACE), (dict(ws_bytes=64), WORKSPACE), (dict(dx=at(0)), INVALID),
    (dict(dres=at(7, 8)), INVALID), (dict(dres=at(1)), INVALID), (dict(dres=at(8)), INVALID), (dict(dw=at(9, 0), dscale=at(9, 4)), INVALID),
    (dict(dw=at(12)), INVALID), (dict(dx=at(7)), INVALID),
])
def test_residual_norm_bwd_refuses(case, status):
    st, msg = residual("bwd", **case)
    assert st == status and msg, (st, msg)


def test_empty_calls_launch_nothing():
    assert gated(seqlen=0)[0] == OK and residual(rows=0)[0] == OK
    assert gated("bwd", seqlen=0, dw=None, ws=None, ws_bytes=0)[0] == OK
    assert residual("bwd", rows=0, dw=None, dw_post=None, dscale=None)[0] == OK
    assert gdr(seqlen=0, h_final=None, ws=None, ws_bytes=0)[0] == OK
    assert gdr("bwd", seqlen=0, dh0=None, ws=None, ws_bytes=0)[0] == OK


def test_sizes():
    assert b.ss_gated_norm_bwd_workspace_bytes(2, 0, 1, 16, 0) == 0 and b.ss_gated_norm_bwd_workspace_bytes(2, 4, 1, 9000, 0) == 0
    assert b.ss_gated_norm_bwd_workspace_bytes(2, 4, 1, 16, 8) == 0
    assert 0 < b.ss_gated_norm_bwd_workspace_bytes(1, (1 << 32) - 1, 1, 8192, 0) < 1 << 30       # bounded, however long the sequence
    assert 0 < b.ss_gated_norm_bwd_workspace_bytes(1, 1 << 11, 1 << 20, 8, b.SS_NORM_HEAD_WEIGHTS) <= 1 << 26
    assert b.ss_residual_norm_bwd_workspace_bytes(0, 16) == 0 and b.ss_residual_norm_bwd_workspace_bytes(5, 9000) == 0
    assert 0 < b.ss_residual_norm_bwd_workspace_bytes((1 << 32) - 1, 8192) < 1 << 30
    assert b.ss_gdr_bwd_workspace_bytes(1, 0, 1, 1, 16, 16) == 0 and b.ss_gdr_bwd_workspace_bytes(1, 5, 2, 3, 16, 16) == 0
    one, two = b.ss_gdr_bwd_workspace_bytes(1, 64, 1, 1, 128, 128), b.ss_gdr_bwd_workspace_bytes(1, 128, 1, 1, 128, 128)
    assert two >= one + 2 * (128 + 64) * 128 * 4           # two states, U and the gradient of R
    assert b.ss_gdr_fwd_workspace_bytes(1, 16, 1, 1, 16, 16) == 0 and b.ss_gdr_fwd_workspace_bytes(1, 17, 1, 1, 16, 16) > 0
    assert b.ss_gdr_fwd_workspace_bytes(0, 5, 1, 1, 16, 16) == 0 and b.ss_gdr_fwd_workspace_bytes(1, 5, 1, 1, 200, 16) == 0
