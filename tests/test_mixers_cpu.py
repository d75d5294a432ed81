"""The gated linear recurrence and the norm and rotation of queries and keys on the CPU: what their C entry
points refuse before they launch anything, and their size queries.

The addresses are made up and only compared; every call here fails its checks or has nothing to launch.
"""
import ctypes

import pytest

from selective_state_space_62_amd import binding as b

BASE = 0x7F0000000000
GB = 1 << 30
OK_IO = b.SS_BF16


def at(k, off=0):
    return BASE + k * GB + off


def glr(entry, **kw):
    a = dict(batch=2, dim=64, seqlen=300, io=OK_IO, kind=b.SS_GLR_NORMALISED, scale=8.0, x=at(0), r=at(1), i=at(2), z=at(3),
             decay=at(4), r_bias=at(5), i_bias=at(6), h0=at(7), y=at(8), h_final=at(9), ckpt=at(10), dy=at(11),
             dh_final=at(12), dx=at(13), dr=at(14), di=at(15), dz=at(16), ddecay=at(17), dr_bias=at(18), di_bias=at(19),
             dh0=at(20), ws=at(21), ws_bytes=1 << 28, state_in=at(22), state_out=at(22))
    a.update(kw)
    ins = [a[k] for k in ("x", "r", "i", "z", "decay", "r_bias", "i_bias")]
    head = [a["batch"], a["dim"], a["seqlen"], a["io"], a["kind"], a["scale"]]
    if entry == "fwd":
        st = b.lib.ss_glr_fwd(*head, *ins, a["h0"], a["y"], a["h_final"], a["ckpt"], a["ws"], a["ws_bytes"], None)
    elif entry == "bwd":
        st = b.lib.ss_glr_bwd(*head, *ins, a["h0"], a["dy"], a["dh_final"], a["ckpt"], a["dx"], a["dr"], a["di"], a["dz"],
                              a["ddecay"], a["dr_bias"], a["di_bias"], a["dh0"], a["ws"], a["ws_bytes"], None)
    else:
        del head[2]
        st = b.lib.ss_glr_step(*head, a["state_in"], a["state_out"], *ins, a["y"], None)
    return st, b.last_error()


INVALID, UNSUPPORTED, WORKSPACE = b.SS_ERR_INVALID_ARG, b.SS_ERR_UNSUPPORTED, b.SS_ERR_WORKSPACE
EVERY = [
    (dict(io=7), UNSUPPORTED), (dict(kind=2), UNSUPPORTED), (dict(kind=-1), UNSUPPORTED), (dict(batch=0), INVALID),
    (dict(dim=0), INVALID), (dict(dim=(1 << 40) + 1), INVALID), (dict(batch=1 << 40, dim=1 << 30), INVALID),
    (dict(x=None), INVALID), (dict(r=None), INVALID), (dict(decay=None), INVALID), (dict(i=None), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(x=at(0, 1)), INVALID), (dict(z=at(3, 1)), INVALID),
    (dict(io=b.SS_F32, r=at(1, 2)), INVALID),
    (dict(decay=at(4, 2)), INVALID), (dict(r_bias=at(5, 1)), INVALID),
]


@pytest.mark.parametrize("case,status", EVERY + [
    (dict(seqlen=-1), INVALID), (dict(y=None), INVALID), (dict(y=at(8, 1)), INVALID), (dict(h0=at(7, 2)), INVALID),
    (dict(h_final=at(9, 2)), INVALID), (dict(ckpt=at(10, 2)), INVALID), (dict(y=at(0)), INVALID),
    (dict(y=at(1, 2 * 64 * 300 * 2 - 16)), INVALID), (dict(h_final=at(7)), INVALID), (dict(ckpt=at(9)), INVALID),
    (dict(h_final=at(8)), INVALID), (dict(dim=1, seqlen=9000, ws=None), WORKSPACE),
    (dict(dim=1, seqlen=9000, ws=at(21, 64)), WORKSPACE), (dict(dim=1, seqlen=9000, ws_bytes=64), WORKSPACE),
    (dict(dim=1, seqlen=9000, h_final=at(21)), INVALID),
])
def test_glr_fwd_refuses(case, status):
    st, msg = glr("fwd", **case)
    assert st == status and msg, (st, msg)


@pytest.mark.parametrize("case,status", EVERY + [
    (dict(seqlen=-1), INVALID), (dict(dy=None), INVALID), (dict(dx=None), INVALID), (dict(dr=None), INVALID),
    (dict(di=None), INVALID), (dict(dz=None), INVALID), (dict(z=None), INVALID),
    (dict(i=None, i_bias=None, di=None), INVALID),                                   # di_bias without i
    (dict(dx=at(13, 1)), INVALID), (dict(dh0=at(20, 2)), INVALID), (dict(dx=at(0)), INVALID), (dict(dr=at(13)), INVALID),
    (dict(ddecay=at(18)), INVALID), (dict(ws=None), WORKSPACE), (dict(ws=at(21, 128)), WORKSPACE),
    (dict(ws_bytes=64), WORKSPACE), (dict(seqlen=5000, ws_bytes=2048), WORKSPACE), (dict(dh0=at(21, 256)), INVALID),
])
def test_glr_bwd_refuses(case, status):
    st, msg = glr("bwd", **case)
    assert st == status and msg, (st, msg)


@pytest.mark.parametrize("case,status", EVERY + [
    (dict(batch=1, dim=(1 << 31) + 1), UNSUPPORTED), (dict(state_in=None), INVALID), (dict(state_out=None), INVALID), (dict(y=None), INVALID), (dict(y=at(0)), INVALID),
    (dict(state_out=at(22, 256)), INVALID), (dict(state_out=at(23, 2)), INVALID), (dict(y=at(22)), INVALID),
])
def test_glr_step_refuses(case, status):
    st, msg = glr("step", **case)
    assert st == status and msg, (st, msg)


def test_glr_convex_needs_no_scale_or_decay():
    """What the convex kind does not read it does not refuse: the next refusal is the workspace's."""
    st, _ = glr("bwd", kind=b.SS_GLR_CONVEX, decay=None, scale=float("nan"), ws=None)
    assert st == WORKSPACE


def test_glr_sizes():
    assert b.ss_glr_ckpt_bytes(2, 3, 2048) == 2 * 3 * 4
    assert b.ss_glr_ckpt_bytes(2, 3, 2049) == 2 * 3 * 2 * 4
    assert b.ss_glr_ckpt_bytes(2, 3, 0) == 0 and b.ss_glr_ckpt_bytes(0, 3, 5) == 0 and b.ss_glr_ckpt_bytes(1, 1, -1) == 0
    assert b.ss_glr_fwd_workspace_bytes(8, 5120, 2048) == 0 and b.ss_glr_fwd_workspace_bytes(1, 2048, 1 << 20) == 0
    # 8 tiles of 2048 tokens and one group of them: a slot each, and a counter
    assert b.ss_glr_fwd_workspace_bytes(1, 10, 16384) == (10 * (8 + 1 + 1) * 8 + 255) // 256 * 256
    assert b.ss_glr_fwd_workspace_bytes(1, 10, 8192) == 0 and b.ss_glr_fwd_workspace_bytes(1, 0, 16384) == 0
    assert b.ss_glr_bwd_workspace_bytes(0, 1, 1) == 0 and b.ss_glr_bwd_workspace_bytes(2, 64, 300) >= 2 * 64 * 3 * 4


def qk(entry="fwd", **kw):
    a = dict(batch=2, seqlen=10, hq=2, hk=1, n=16, rot=16, io=OK_IO, flags=0, eps=1e-6, q=at(0), qs=(480, 48, 16), k=at(0, 64),
             ks=(480, 48, 16), wq=at(1), wk=at(2), freq=at(3), pos=at(4), pos0=0, qo=at(5), ko=at(6), dqo=at(7), dko=at(8),
             dq=at(9), dqs=(320, 32, 16), dk=at(10), dks=(160, 16, 16), dwq=at(11), dwk=at(12), ws=at(13), ws_bytes=1 << 24)
    a.update(kw)
    head = [a["batch"], a["seqlen"], a["hq"], a["hk"], a["n"], a["rot"], a["io"], a["flags"], a["eps"], a["q"],
            b._strides(a["qs"]), a["k"], b._strides(a["ks"]), a["wq"], a["wk"], a["freq"], a["pos"], a["pos0"]]
    if entry == "fwd":
        st = b.lib.ss_qk_norm_rot(*head, a["qo"], a["ko"], None)
    else:
        st = b.lib.ss_qk_norm_rot_bwd(*head, a["dqo"], a["dko"], a["dq"], b._strides(a["dqs"]), a["dk"],
                                      b._strides(a["dks"]), a["dwq"], a["dwk"], a["ws"], a["ws_bytes"], None)
    return st, b.last_error()


COMMON = [
    (dict(io=3), UNSUPPORTED), (dict(flags=4), UNSUPPORTED), (dict(batch=0), INVALID), (dict(seqlen=-1), INVALID),
    (dict(hq=-1), INVALID), (dict(hq=0, hk=0), INVALID), (dict(hq=(1 << 20) + 1), INVALID), (dict(n=0), UNSUPPORTED),
    (dict(n=257), UNSUPPORTED), (dict(n=24, rot=16, flags=b.SS_QK_FEATURE_MAJOR), UNSUPPORTED), (dict(rot=-2), INVALID),
    (dict(rot=3), INVALID), (dict(rot=18), INVALID), (dict(eps=0.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(eps=1e-40), INVALID), (dict(freq=None), INVALID), (dict(freq=at(3, 4)), INVALID), (dict(pos=at(4, 4)), INVALID),
    (dict(wq=at(1, 2)), INVALID), (dict(wk=at(2, 1)), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID),
    (dict(hk=0), INVALID), (dict(q=at(0, 1)), INVALID), (dict(qs=(480, -48, 16)), INVALID), (dict(ks=None), INVALID),
    (dict(qs=(1 << 62, 48, 16)), INVALID), (dict(batch=1 << 40, seqlen=1 << 30), INVALID),
]


@pytest.mark.parametrize("case,status", COMMON + [
    (dict(qo=None), INVALID), (dict(ko=None), INVALID), (dict(qo=at(5, 8)), INVALID), (dict(qo=at(0)), INVALID),
    (dict(ko=at(0, 96)), INVALID), (dict(ko=at(5, 64)), INVALID), (dict(qo=at(4)), INVALID), (dict(hk=0, k=None), INVALID),
])
def test_qk_norm_rot_refuses(case, status):
    st, msg = qk(**case)
    assert st == status and msg, (st, msg)


@pytest.mark.parametrize("case,status", COMMON + [
    (dict(dqo=None), INVALID), (dict(dko=at(8, 4)), INVALID), (dict(dq=None), INVALID), (dict(dk=at(10, 1)), INVALID),
    (dict(dqs=(320, 32, 8)), INVALID),                  # heads share values
    (dict(dqs=(320, 16, 16)), INVALID),                 # tokens share values
    (dict(dqs=(32, 32, 16)), INVALID),                  # batch rows share values
    (dict(dqs=(0, 32, 16)), INVALID), (dict(dk=at(9)), INVALID),
    (dict(dk=at(9, 62), dqs=(480, 48, 16), dks=(480, 48, 16)), INVALID),        # the first column of dk is the last of dq
    (dict(dk=at(9, 66), dqs=(480, 48, 16), dks=(480, 48, 16)), INVALID),        # dk ends in the next row
    (dict(dk=at(9, 64), dqs=(480, 48, 16), dks=(960, 96, 16)), INVALID),        # other rows
    (dict(dq=at(0, 96 * 5)), INVALID), (dict(dwq=at(12)), INVALID), (dict(dwq=at(11, 2)), INVALID), (dict(dwk=at(13)), INVALID),
    (dict(ws=None), WORKSPACE), (dict(ws=at(13, 16)), WORKSPACE), (dict(ws_bytes=16), WORKSPACE),
    (dict(hk=0, k=None, dko=None, dk=None), INVALID),   # dwk of no keys
])
def test_qk_norm_rot_bwd_refuses(case, status):
    st, msg = qk("bwd", **case)
    assert st == status and msg, (st, msg)


def test_gradient_columns_of_one_buffer_pass_the_overlap_check():
    """dq and dk side by side in rows of 48: only the workspace is refused."""
    st, msg = qk("bwd", dk=at(9, 64), dqs=(480, 48, 16), dks=(480, 48, 16), ws=None)
    assert st == WORKSPACE, msg
    st, msg = qk("bwd", dq=at(9, 32), dk=at(9), dqs=(480, 48, 16), dks=(480, 48, 16), ws_bytes=16)
    assert st == WORKSPACE, msg


def test_qk_empty_sequence_launches_nothing():
    assert qk(seqlen=0)[0] == b.SS_OK
    assert qk("bwd", seqlen=0, dwq=None, dwk=None, ws=None, ws_bytes=0)[0] == b.SS_OK


def test_qk_sizes():
    assert b.ss_qk_norm_rot_bwd_workspace_bytes(2, 0, 1, 1, 16) == 0
    assert b.ss_qk_norm_rot_bwd_workspace_bytes(2, 10, 0, 0, 16) == 0
    assert b.ss_qk_norm_rot_bwd_workspace_bytes(2, 10, 1, 1, 300) == 0
    n = b.ss_qk_norm_rot_bwd_workspace_bytes(1, 1 << 40, 1, 1, 256)
    assert 0 < n < 1 << 30      # bounded, however long the sequence


@pytest.mark.parametrize("entry", ["fwd", "bwd"])
@pytest.mark.parametrize("pos0", [(1 << 53) - 9, (1 << 63) - 1, -(1 << 53) - 1, -(1 << 63)])
def test_positions_past_fp64(entry, pos0):
    """pos0 + t of ten tokens beyond 2^53, where fp64 holds no odd position and 64 bits end; given positions are used instead of it."""
    st, msg = qk(entry, pos=None, pos0=pos0)
    assert st == INVALID and "pos0" in msg, (st, msg)
    assert "pos0" not in qk(entry, pos0=pos0, qo=None, dqo=None)[1]
    assert "pos0" not in qk(entry, pos=None, pos0=(1 << 53) - 10, qo=None, dqo=None)[1]


def test_strides_marshal():
    assert b._strides(None) is None
    assert list(b._strides((1, 2, 3))) == [1, 2, 3] and isinstance(b._strides((1, 2, 3)), ctypes.Array)


# dq and dk in one buffer without a shared address: (dq's strides, dk's strides, dk's elements after dq), 2 heads and 1 unless given
INTERLEAVED = [
    (dict(hq=4, hk=4), (1920, 192, 48), (1920, 192, 48), 16),        # (batch, token, head, [q k v]): heads alternate
    (dict(hq=4, hk=4), (1920, 192, 48), (1920, 192, 48), -16),       # [k q v]
    (dict(hq=4, hk=4), (1280, 128, 32), (1280, 128, 32), 16),        # [q k], nothing between
    (dict(hq=4, hk=1), (800, 80, 16), (800, 80, 16), -16),           # the key's columns first, the last head's end the row's
    (dict(hq=1, hk=3), (960, 96, 16), (960, 96, 32), 16),            # one query before three keys 32 apart
    ({}, (48, 96, 16), (48, 96, 16), 32),                            # (token, batch, columns)
    (dict(hq=4, hk=4), (192, 384, 48), (192, 384, 48), 16),          # (token, batch, head, [q k v])
    (dict(hq=3, hk=3), (1280, 16, 320), (1280, 16, 320), 160),       # (batch, head, [q k], token)
    (dict(seqlen=1), (48, 0, 16), (48, 0, 16), 32),
    (dict(batch=1, hq=2, hk=2), (0, 64, 32), (7, 64, 32), 16),       # a batch of one has no stride
]


@pytest.mark.parametrize("sizes,dqs,dks,apart", INTERLEAVED)
def test_interleaved_gradients_pass_the_overlap_check(sizes, dqs, dks, apart):
    """Only dwk is refused, which lies on the workspace and is looked at after dq and dk; and by counting, no two values share an
    address."""
    st, msg = qk("bwd", dq=at(9, 1024), dk=at(9, 1024 + 2 * apart), dqs=dqs, dks=dks, dwk=at(13), **sizes)
    assert st == INVALID and "dwk overlaps workspace" in msg, (st, msg)
    assert _shared(dict(dict(batch=2, seqlen=10, hq=2, hk=1), **sizes), dqs, dks, apart) == 0


def _shared(sizes, dqs, dks, apart):
    import numpy as np
    seen = []
    for heads, s, off in ((sizes["hq"], dqs, 0), (sizes["hk"], dks, apart)):
        b, t, h, j = np.ogrid[:sizes["batch"], :sizes["seqlen"], :heads, :16]
        seen.append((off + b * s[0] + t * s[1] + h * s[2] + j).ravel())
    seen = np.concatenate(seen)
    return seen.size - np.unique(seen).size


@pytest.mark.parametrize("sizes,dqs,dks,apart", [
    (dict(hq=4, hk=4), (1920, 192, 48), (1920, 192, 48), 8),         # half a vector shared
    (dict(hq=4, hk=4), (1920, 192, 48), (1920, 192, 48), 40),        # into the next head
    (dict(hq=4, hk=4), (1920, 192, 48), (1920, 192, 48), 48),        # the next head itself
    (dict(hq=4, hk=4), (1920, 192, 48), (1920, 192, 48), 176 + 8),   # into the next token
    (dict(hq=4, hk=4), (192, 384, 48), (192, 384, 48), 192),         # the other batch row
    (dict(hq=1, hk=3), (960, 96, 16), (960, 96, 32), 32 + 8),
    (dict(hq=3, hk=3), (1280, 16, 320), (1280, 16, 320), 144),
    (dict(seqlen=1), (48, 0, 16), (48, 0, 16), 24),
])
def test_shared_gradients_are_refused(sizes, dqs, dks, apart):
    assert _shared(dict(dict(batch=2, seqlen=10, hq=2, hk=1), **sizes), dqs, dks, apart) > 0
    st, msg = qk("bwd", dq=at(9, 1024), dk=at(9, 1024 + 2 * apart), dqs=dqs, dks=dks, **sizes)
    assert st == INVALID and "overlaps dk" in msg, (st, msg)


@pytest.mark.parametrize("dim", [(1 << 31) - 127, 1 << 31])
def test_glr_step_refuses_more_channels_than_a_grid(dim):
    """A workgroup takes 128 channels and a grid dimension has fewer than 2^32 threads, so fewer than 2^24 of its workgroups."""
    st, msg = glr("step", batch=1, dim=dim)
    assert st == UNSUPPORTED and "dim" in msg, (st, msg)
    st, msg = glr("step", batch=1, dim=(1 << 31) - 128, y=None)
    assert st == INVALID and "y is NULL" in msg, (st, msg)


@pytest.mark.parametrize("batch,dim,L,io", [(33, 5, 37, "f32"), (2, 3, 6145, "f32"), (40, 3, 2048 * 7 + 5, "bf16")])
def test_a_lost_term_would_show_in_the_counted_sums(batch, dim, L, io):
    """The inputs of the recurrence's sums over tokens: no term is 0 where the gate is not, each is exact in fp32, and the sum of their
    sizes is too, so that fp32 sums of them in any order are exact and one term less is another value."""
    import numpy as np
    import torch
    from test_gpu_glr import counted
    p, _, terms = counted(torch.device("cpu"), batch, dim, L, io)
    for k, v in terms.items():
        shown = v[..., 1::2] if k == "dr_bias" else v
        assert (shown != 0).all() and np.array_equal(v.astype(np.float32), v), k
        assert (v * 16 == np.rint(v * 16)).all() and np.abs(v).sum((0, 2)).max() < 2 ** 20, k
    assert p["x"].dtype == (torch.float32 if io == "f32" else torch.bfloat16)
