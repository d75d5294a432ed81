"""The norm and rotation of queries and keys on the GPU against the formulas in 64 bits."""
import numpy as np
import pytest

from gpu_util import log, to_f64

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {"f32": U, "bf16": 2.0 ** -8}
EPS = 1e-6


@pytest.fixture(scope="module")
def dev():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return torch.device("cuda:0")


@pytest.fixture(scope="module")
def ss():
    import selective_state_space_62_amd as m
    return m


def rotate(n, pos, freq, interleaved, back=False):
    """n (B, L, H, N) with its first 2 len(freq) values rotated, as complex numbers in 64 bits."""
    R = 2 * len(freq)
    turn = np.exp((-1j if back else 1j) * pos[..., None, None].astype(np.float64) * freq)
    out = n.copy()
    i1, i2 = (np.arange(0, R, 2), np.arange(1, R, 2)) if interleaved else (np.arange(R // 2), np.arange(R // 2, R))
    c = (n[..., i1] + 1j * n[..., i2]) * turn
    out[..., i1], out[..., i2] = c.real, c.imag
    return out


def pair_size(n, freq, interleaved):
    """For each value, the size of the pair it is in (its own where it is not rotated)."""
    R = 2 * len(freq)
    out = np.abs(n).copy()
    i1, i2 = (np.arange(0, R, 2), np.arange(1, R, 2)) if interleaved else (np.arange(R // 2), np.arange(R // 2, R))
    out[..., i1] = out[..., i2] = np.abs(n[..., i1]) + np.abs(n[..., i2])
    return out


def forward(v, w, pos, freq, interleaved):
    """(outputs, fp32 bound).  rho: N products and sums (a tree of at most N + 8), a division, a root; then two products:
    relative N/2 + 12 halves at most.  A rotated value mixes its pair with cos and sin that are each within
    4 halves (octant angle 1, polynomial 2, its rounding 1), two products, a sum; angles in fp64 add |angle| 2^-51."""
    N = v.shape[-1]
    rho = 1.0 / np.sqrt((v * v).mean(-1, keepdims=True) + EPS)
    n = v * rho * (1.0 if w is None else w)
    size = pair_size(n, freq, interleaved)
    far = np.abs(pos[..., None, None]).max(initial=0) * 2.0 ** -51
    return rotate(n, pos, freq, interleaved), size * (U * (N / 2 + 24) + far)


def backward(v, w, pos, freq, interleaved, do):
    N = v.shape[-1]
    ww = np.ones(N) if w is None else w
    rho = 1.0 / np.sqrt((v * v).mean(-1, keepdims=True) + EPS)
    dn = rotate(do, pos, freq, interleaved, back=True)
    far = np.abs(pos[..., None, None]).max(initial=0) * 2.0 ** -51
    edn = pair_size(do, freq, interleaved) * (8 * U + far)
    p = dn * ww
    mean = (p * v).mean(-1, keepdims=True)
    dv = rho * (p - v * rho * rho * mean)
    # of each term: rho's N/2 + 12 halves (thrice in the second), the mean's N + 8, a few products
    emean = (edn * np.abs(ww * v)).mean(-1, keepdims=True) + U * (N + 8) * np.abs(p * v).mean(-1, keepdims=True)
    e = rho * (edn * np.abs(ww) + np.abs(v) * rho * rho * emean) + U * rho * (
        (N / 2 + 16) * np.abs(p) + (1.5 * N + 48) * np.abs(v) * rho * rho * np.abs(mean))
    part = dn * v * rho
    # a value passes at most 64 + tokens * heads / 64 sums or so
    count = v.shape[0] * v.shape[1] * v.shape[2]
    edw = (edn * np.abs(v) * rho + U * (N / 2 + 80 + count / 16) * np.abs(part)).sum((0, 1, 2))
    return dv, e, part.sum((0, 1, 2)), edw


def near(name, got, want, e, half):
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    tol = 2 * e + 1.0001 * half * np.abs(want) + 1e-37
    off = np.abs(got - want)
    assert (off <= tol).all(), "%s: %d of %d outside, worst %.3g of the bound" % (
        name, int((~(off <= tol)).sum()), off.size, float(np.nanmax(off / tol)))


def problem(dev, seed, B, L, hq, hk, N, rot, io="bf16", extra=0, far=False, weights=True):
    """q and k cut from one tensor of rows with `extra` columns before them."""
    import torch
    gen = torch.Generator().manual_seed(seed)
    dt = torch.float32 if io == "f32" else torch.bfloat16
    rows = torch.randn((B, L, extra + (hq + hk) * N), generator=gen).to(dt).to(dev)
    q = rows[..., extra:extra + hq * N].unflatten(-1, (hq, N)) if hq else None
    k = rows[..., extra + hq * N:].unflatten(-1, (hk, N)) if hk else None
    freq = (10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / max(1, rot // 2))).to(dev)
    pos = torch.randint(-(1 << 20), 1 << 20, (B, L), generator=gen).to(dev) if far else None
    w = [1 + 0.3 * torch.randn(N, generator=gen).to(dev) if weights and h else None for h in (hq, hk)]
    return dict(q=q, k=k, inv_freq=freq, wq=w[0], wk=w[1], positions=pos)


def sides(p):
    """(name, input, weight) of the sides that are there, in 64 bits."""
    return [(s, to_f64(p[s]), None if p["w" + s] is None else to_f64(p["w" + s])) for s in ("q", "k") if p[s] is not None]


def where(p, B, L, pos0=0):
    return p["positions"].cpu().numpy() if p["positions"] is not None else np.broadcast_to(pos0 + np.arange(L), (B, L))


def grads_like(dev, seed, p, feature_major):
    import torch
    gen = torch.Generator().manual_seed(seed)

    def like(t):
        if t is None:
            return None
        g = torch.randn(t.shape, generator=gen).to(t.dtype).to(dev)
        return g.permute(0, 2, 3, 1).contiguous() if feature_major else g
    return like(p["q"]), like(p["k"])


def run_both(ss, dev, p, B, L, io, interleaved, feature_major):
    """Forward and backward of one problem, checked."""
    import torch
    pos, freq = where(p, B, L), p["inv_freq"].cpu().numpy()
    kw = dict(interleaved=interleaved, feature_major=feature_major)
    got = dict(zip("qk", ss.qk_norm_rot(**p, **kw)))
    dq, dk = grads_like(dev, 9, p, feature_major)
    back = ss.qk_norm_rot_bwd(dq_out=dq, dk_out=dk, **p, **kw)
    torch.cuda.synchronize()
    for s, v, w in sides(p):
        o, e = forward(v, w, pos, freq, interleaved)
        g = to_f64(got[s])
        near(s, np.moveaxis(g, 3, 1) if feature_major else g, o, e, HALF[io])
        do = to_f64(dq if s == "q" else dk)
        do = np.moveaxis(do, 3, 1) if feature_major else do
        dv, e, dw, edw = backward(v, w, pos, freq, interleaved, do)
        near("d" + s, to_f64(back["d" + s]), dv, e, HALF[io])
        near("dw" + s, to_f64(back["dw" + s]), dw, edw, 0.0)
    return got, back


# (heads_q, heads_k, N, rot): shared heads, one side only, odd dims, part rotated, none rotated, one value
TOKEN_MAJOR = [(4, 2, 64, 64), (1, 1, 16, 16), (5, 1, 80, 32), (3, 3, 128, 128), (2, 0, 256, 256), (0, 2, 72, 72), (2, 1, 33, 10),
               (1, 1, 1, 0), (3, 1, 2, 2), (1, 2, 255, 254), (6, 2, 96, 0), (40, 8, 8, 8), (2, 2, 192, 64), (1, 1, 40, 40)]


@pytest.mark.parametrize("hq,hk,N,rot", TOKEN_MAJOR)
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,L,extra,far", [(1, 1, 0, False), (2, 67, 24, True), (3, 5, 7, False)])
def test_token_major(ss, dev, B, L, extra, far, interleaved, io, hq, hk, N, rot):
    run_both(ss, dev, problem(dev, N + L, B, L, hq, hk, N, rot, io, extra, far), B, L, io, interleaved, False)


@pytest.mark.parametrize("hq,hk,N,rot", [(1, 1, 16, 16), (2, 1, 16, 8), (1, 0, 8, 8), (1, 1, 4, 2), (0, 3, 2, 2), (1, 1, 1, 0), (2, 2, 16, 0)])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,L,extra,far", [(5, 1, 160, True), (2, 67, 7, False), (1, 300, 8, True), (3, 64, 0, False)])
def test_feature_major(ss, dev, B, L, extra, far, interleaved, io, hq, hk, N, rot):
    run_both(ss, dev, problem(dev, N + L, B, L, hq, hk, N, rot, io, extra, far), B, L, io, interleaved, True)


@pytest.mark.parametrize("feature_major", [False, True])
def test_many_tokens(ss, dev, feature_major):
    """More tokens than any plan's workgroups take in one round."""
    run_both(ss, dev, problem(dev, 3, 3, 20011, 1, 1, 16, 16, "bf16", 16, True), 3, 20011, "bf16", False, feature_major)
    if not feature_major:
        run_both(ss, dev, problem(dev, 4, 2, 4099, 8, 2, 64, 64, "bf16"), 2, 4099, "bf16", False, False)


def test_shapes_of_one_head(ss, dev):
    """(batch, L, N) and (batch, N) inputs, and the layouts that the scan and the decode step take."""
    import torch
    p = problem(dev, 5, 4, 9, 1, 1, 16, 16, "bf16", 3)
    q4, k4 = ss.qk_norm_rot(**p, feature_major=True)
    flat = {**p, "q": p["q"][:, :, 0], "k": p["k"][:, :, 0]}
    q3, k3 = ss.qk_norm_rot(**flat, feature_major=True)
    assert q3.shape == (4, 16, 9) and torch.equal(q3, q4[:, 0]) and torch.equal(k3, k4[:, 0])
    for t in (0, 8):
        one = {**p, "q": p["q"][:, t, 0], "k": p["k"][:, t, 0]}
        for fm in (False, True):
            q2, k2 = ss.qk_norm_rot(**{**one, "positions": torch.full((4,), t, device=dev)}, feature_major=fm)
            assert q2.shape == (4, 16) and torch.equal(q2, q3[..., t]) and torch.equal(k2, k3[..., t])
        q2, _ = ss.qk_norm_rot(**one, pos0=t)
        assert torch.equal(q2, q3[..., t])
    torch.cuda.synchronize()


@pytest.mark.parametrize("fm", [False, True])
def test_far_and_negative_positions(ss, dev, fm):
    """Positions of 2^40: the angle's own fp64 rounding, 2^40 * 2^-51 radians, is what is left."""
    import torch
    p = problem(dev, 6, 1, 6, 1, 1, 16, 16, "f32")
    p["positions"] = torch.tensor([[0, -1, (1 << 31) + 1, 1 << 33, -(1 << 40), 1 << 40]], device=dev)
    run_both(ss, dev, p, 1, 6, "f32", False, fm)
    far = ss.qk_norm_rot(**{**p, "positions": None}, pos0=(1 << 35) - 3, feature_major=fm)
    given = ss.qk_norm_rot(**{**p, "positions": torch.arange(6, device=dev)[None] + (1 << 35) - 3}, feature_major=fm)
    torch.cuda.synchronize()
    assert torch.equal(far[0], given[0]) and torch.equal(far[1], given[1])


def test_zero_infinite_and_nan_vectors(ss, dev):
    """A vector of zeros gives zeros and finite gradients; one of NaN or infinity spoils itself alone."""
    import torch
    for N, fm in ((64, False), (16, True)):
        p = problem(dev, 7, 1, 8, 2, 1, N, N, "f32")
        clean = ss.qk_norm_rot(**p, feature_major=fm)[0].clone()
        p["q"][0, 2] = 0
        p["q"][0, 4, 1, 3] = float("nan")
        p["q"][0, 6, 0, 5] = float("inf")
        out = ss.qk_norm_rot(**p, feature_major=fm)[0]
        do = torch.ones_like(out)
        g = ss.qk_norm_rot_bwd(p["q"], None, p["inv_freq"], do, None, wq=p["wq"], feature_major=fm)
        torch.cuda.synchronize()
        if fm:
            out, clean = out.permute(0, 3, 1, 2), clean.permute(0, 3, 1, 2)
        assert not out[0, 2].any() and torch.isfinite(g["dq"][0, 2]).all()
        assert torch.isnan(out[0, 4, 1]).all() and torch.isnan(out[0, 6, 0]).any()
        for t, h in ((0, 0), (4, 0), (6, 1), (7, 1)):
            assert torch.equal(out[0, t, h], clean[0, t, h])


def test_gradient_into_columns_of_one_buffer(ss, dev):
    import torch
    for fm, N, hq, hk in ((True, 16, 1, 1), (False, 40, 3, 2)):
        p = problem(dev, 8, 2, 33, hq, hk, N, N, "bf16", 8)
        dq, dk = grads_like(dev, 10, p, fm)
        want = ss.qk_norm_rot_bwd(dq_out=dq, dk_out=dk, **p, feature_major=fm)
        rows = torch.full((2, 33, 8 + (hq + hk) * N + 5), 7.0, dtype=torch.bfloat16, device=dev)
        gk = rows[..., 8:8 + hk * N].unflatten(-1, (hk, N))
        gq = rows[..., 8 + hk * N:8 + (hq + hk) * N].unflatten(-1, (hq, N))
        got = ss.qk_norm_rot_bwd(dq_out=dq, dk_out=dk, **p, feature_major=fm, dq=gq, dk=gk)
        torch.cuda.synchronize()
        assert got["dq"] is gq and torch.equal(gq, want["dq"]) and torch.equal(gk, want["dk"])
        assert (rows[..., :8] == 7).all() and (rows[..., 8 + (hq + hk) * N:] == 7).all()


@pytest.mark.parametrize("fm,N,hq,hk", [(True, 16, 1, 1), (False, 64, 2, 1), (False, 7, 1, 1)])
def test_offsets_past_32_bits(ss, dev, fm, N, hq, hk):
    """Rows whose last ones start more than 2^31 elements on: as from contiguous copies, gradients into such rows too."""
    import torch
    B, L, width = 2, 1100, 1 << 20
    p = problem(dev, 16, B, L, hq, hk, N, N // 2 * 2, "bf16")
    rows = torch.empty(B, L, width, dtype=torch.bfloat16, device=dev)
    n = (hq + hk) * N
    wide = rows[..., -n:]
    far = dict(p, q=wide[..., :hq * N].unflatten(-1, (hq, N)), k=wide[..., hq * N:].unflatten(-1, (hk, N)))
    far["q"].copy_(p["q"])
    far["k"].copy_(p["k"])
    want, got = ss.qk_norm_rot(**p, feature_major=fm), ss.qk_norm_rot(**far, feature_major=fm)
    dq, dk = grads_like(dev, 17, p, fm)
    gw = ss.qk_norm_rot_bwd(dq_out=dq, dk_out=dk, **p, feature_major=fm)
    grad = torch.empty_like(rows)
    dst = [grad[..., a:a + h * N].unflatten(-1, (h, N)) for a, h in ((0, hq), (hq * N, hk))]
    gg = ss.qk_norm_rot_bwd(dq_out=dq, dk_out=dk, **far, feature_major=fm, dq=dst[0], dk=dst[1])
    torch.cuda.synchronize()
    for a, b in ((want[0], got[0]), (want[1], got[1]), *((gw[k], gg[k]) for k in gw)):
        assert torch.equal(a, b)


def test_broadcast_inputs(ss, dev):
    """One row shared by all tokens (stride 0) and heads apart by more than their values."""
    import torch
    wide = torch.randn(1, 1, 4, 96, device=dev)
    q = wide[..., :64].expand(3, 20, 4, 64)
    freq = torch.linspace(0.5, 0.01, 32, dtype=torch.float64, device=dev)
    a, _ = ss.qk_norm_rot(q, None, freq)
    b, _ = ss.qk_norm_rot(q.contiguous(), None, freq)
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_repeats_and_graph_replays_are_bitwise_equal(ss, dev):
    import torch
    for fm, N, hq in ((True, 16, 1), (False, 64, 4)):
        p = problem(dev, 11, 2, 500, hq, 1, N, N, "bf16", 16)
        dq, dk = grads_like(dev, 12, p, fm)

        def both():
            q, k = ss.qk_norm_rot(**p, feature_major=fm)
            return dict(ss.qk_norm_rot_bwd(dq_out=dq, dk_out=dk, **p, feature_major=fm), q=q, k=k)

        want = {n: v.clone() for n, v in both().items()}
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            both()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = both()
        for k in range(3):
            for v in got.values():
                v.zero_()
            g.replay()
            torch.cuda.synchronize()
            again = both()
            torch.cuda.synchronize()
            for n in want:
                assert torch.equal(got[n], want[n]) and torch.equal(again[n], want[n]), (n, k)


def test_gradients_against_differences():
    """The formulas' gradients, which the kernels are held to above, against central differences in 64 bits."""
    rng = np.random.default_rng(3)
    B, L, H, N = 1, 3, 2, 6
    v, w, do = rng.standard_normal((B, L, H, N)), rng.standard_normal(N), rng.standard_normal((B, L, H, N))
    pos, freq = rng.integers(0, 50, (B, L)), np.array([1.0, 0.1])
    for inter in (False, True):
        dv, _, dw, _ = backward(v, w, pos, freq, inter, do)
        loss = lambda v, w: float((forward(v, w, pos, freq, inter)[0] * do).sum())  # noqa: E731
        for x, g, f in ((v, dv, lambda t: loss(t, w)), (w, dw, lambda t: loss(v, t))):
            for at in np.ndindex(x.shape):
                up, dn = x.copy(), x.copy()
                up[at] += 1e-6
                dn[at] -= 1e-6
                assert abs((f(up) - f(dn)) / 2e-6 - g[at]) < 1e-7


def test_rotated_scan_is_a_complex_recurrence(ss, dev):
    """B and C normed and rotated into the scan: with the decays shared by a pair, each pair of states is one complex state
    whose readout sees only the distance between tokens."""
    import torch
    B, L, D, N, extra = 2, 150, 12, 16, 20
    p = problem(dev, 13, B, L, 1, 1, N, N, "f32", extra)
    gen = torch.Generator().manual_seed(2)
    x, dt = (torch.randn(B, D, L, generator=gen).to(dev) for _ in range(2))
    A = -(torch.rand(D, N // 2, generator=gen) + 0.1).repeat(1, 2).to(dev)      # pairs (j, j + N/2) share it
    C, Bm = ss.qk_norm_rot(p["q"][:, :, 0], p["k"][:, :, 0], p["inv_freq"], p["wq"], p["wk"], pos0=1 << 20, feature_major=True)
    y, _ = ss.scan_fwd(x, dt, Bm, C, A)
    torch.cuda.synchronize()

    def normed(v, w):
        v = to_f64(v)[:, :, 0]
        n = v / np.sqrt((v * v).mean(-1, keepdims=True) + EPS) * to_f64(w)
        return n[..., :N // 2] + 1j * n[..., N // 2:]
    q, k = normed(p["q"], p["wq"]), normed(p["k"], p["wk"])
    delta = np.logaddexp(0.0, to_f64(dt))
    freq, a, xs = to_f64(p["inv_freq"]), to_f64(A)[:, :N // 2], to_f64(x)
    h, want = np.zeros((B, D, N // 2), complex), np.empty((B, D, L))
    for t in range(L):
        h = np.exp(delta[..., t, None] * a - 1j * freq) * h + (delta[..., t] * xs[..., t])[..., None] * k[:, None, t]
        want[..., t] = (np.conj(q[:, None, t]) * h).sum(-1).real
    e = np.linalg.norm(to_f64(y) - want) / np.linalg.norm(want)
    log("rotated scan against the complex recurrence: rel-L2 %.2e" % e)
    assert e < 1e-5


def test_a_stack_of_mixers_decodes_as_it_prefills(ss, dev):
    """Norm and rotation into the scan, the scan's output into the gated linear recurrence: whole sequence against one
    token at a time, and the gradients handed back along the same path."""
    import torch
    B, L, D, N = 3, 70, 40, 16
    p = problem(dev, 14, B, L, 1, 1, N, N, "f32", 4)
    gen = torch.Generator().manual_seed(8)
    x, dt, r, i, z = (torch.randn(B, D, L, generator=gen).to(dev) for _ in range(5))
    A = -(torch.rand(D, N, generator=gen) + 0.1).to(dev)
    decay = (torch.rand(D, generator=gen) * 4 - 4).to(dev)
    rot = dict(inv_freq=p["inv_freq"], wq=p["wq"], wk=p["wk"], feature_major=True)
    gates = dict(decay=decay, kind="normalised")
    C, Bm = ss.qk_norm_rot(p["q"][:, :, 0], p["k"][:, :, 0], **rot)
    y1, h1 = ss.scan_fwd(x, dt, Bm, C, A)
    y2, h2 = ss.glr_fwd(y1, r, i, z, **gates)
    s1, s2 = torch.zeros(B, D, N, device=dev), torch.zeros(B, D, device=dev)
    for t in range(L):
        c, b = ss.qk_norm_rot(p["q"][:, t, 0], p["k"][:, t, 0], pos0=t, **rot)
        o = ss.state_update(s1, x[..., t].contiguous(), dt[..., t].contiguous(), b, c, A)
        o = ss.glr_step(s2, o, *(v[..., t].contiguous() for v in (r, i, z)), **gates)
        assert float((o - y2[..., t]).abs().max()) <= 1e-4 * float(y2.abs().max()), t
    assert float((s2 - h2).abs().max()) <= 1e-4 * float(h2.abs().max())
    dy = torch.randn(B, D, L, generator=gen).to(dev)
    g2 = ss.glr_bwd(y1, r, dy, i, z, **gates)
    g1 = ss.scan_bwd(x, dt, Bm, C, A, g2["dx"])
    g0 = ss.qk_norm_rot_bwd(p["q"][:, :, 0], p["k"][:, :, 0], p["inv_freq"], g1["dC"], g1["dB"], wq=p["wq"], wk=p["wk"],
                            feature_major=True)
    torch.cuda.synchronize()
    # along a random direction of q and k: the change of the loss against the gradients' product with it.  fp32 losses of
    # about 1e3 terms carry 1e-5 relative; a step of 1e-2 has a second difference of 1e-4 of them
    for name in ("q", "k"):
        v = torch.randn(p[name].shape, generator=gen).to(dev)
        v *= 1e-2
        losses = []
        for sign in (1.0, -1.0):
            q, k = (p[s] + sign * v if s == name else p[s] for s in ("q", "k"))
            C, Bm = ss.qk_norm_rot(q[:, :, 0], k[:, :, 0], **rot)
            losses.append(float((ss.glr_fwd(ss.scan_fwd(x, dt, Bm, C, A)[0], r, i, z, **gates)[0] * dy).double().sum()))
        want = float((g0["d" + name] * v[:, :, 0]).double().sum())
        size = float((g0["d" + name].double().norm() * v.double().norm()))
        assert abs((losses[0] - losses[1]) / 2 - want) <= 1e-2 * size, (name, losses, want, size)


def test_tensor_checks(ss, dev):
    import torch
    p = problem(dev, 15, 2, 4, 2, 1, 64, 64, "bf16")
    for change, err in ((dict(k=p["k"].float()), TypeError), (dict(k=p["k"][:, :3]), ValueError), (dict(k=p["k"][..., :32]), ValueError),
                        (dict(q=p["q"][..., ::2], k=None), ValueError), (dict(inv_freq=p["inv_freq"].float()), TypeError),
                        (dict(inv_freq=torch.ones(33, dtype=torch.float64, device=dev)), ss.SsError), (dict(wq=p["wq"][:8]), ValueError),
                        (dict(positions=torch.zeros(2, 4, dtype=torch.int32, device=dev)), TypeError), (dict(q=None, k=None), ValueError),
                        (dict(feature_major=True), ss.SsError), (dict(eps=0.0), ss.SsError), (dict(q=p["q"].cpu(), k=None), ValueError),
                        (dict(q_out=torch.empty(2, 4, 2, 63, dtype=torch.bfloat16, device=dev)), ValueError)):
        with pytest.raises(err):
            ss.qk_norm_rot(**{**p, **change})
    dq, dk = grads_like(dev, 1, p, False)
    with pytest.raises(ValueError):
        ss.qk_norm_rot_bwd(dq_out=dq[:, :3], dk_out=dk, **p)
    with pytest.raises(ss.SsError):
        shared = torch.empty(2, 4, 1, 64, dtype=torch.bfloat16, device=dev).expand(2, 4, 2, 64)
        ss.qk_norm_rot_bwd(dq_out=dq, dk_out=dk, dq=shared, **p)


@pytest.mark.parametrize("pos0", [1 << 64, -(1 << 63) - 1, (1 << 64) + 5])
def test_pos0_of_more_than_64_bits_is_refused(ss, dev, pos0):
    p = problem(dev, 18, 1, 4, 1, 1, 16, 16, "f32")
    p["positions"] = None
    with pytest.raises(ValueError):
        ss.qk_norm_rot(**p, pos0=pos0)
    with pytest.raises(ValueError):
        ss.qk_norm_rot_bwd(dq_out=p["q"], dk_out=p["k"], **p, pos0=pos0)
    with pytest.raises(ss.SsError):
        ss.qk_norm_rot(**p, pos0=1 << 60)


@pytest.mark.parametrize("fm,N,order", [(False, 40, "b t h s"), (True, 16, "b t h s"), (False, 64, "t b h s"), (False, 33, "b h s t")])
def test_gradient_between_the_heads_of_one_buffer(ss, dev, fm, N, order):
    """q, k and v of a head side by side, head after head, batch row or token first: inputs and gradients there are those of
    contiguous ones, and what lies at v is left alone."""
    import torch
    size = dict(b=2, t=37, h=3, s=3)
    axes = order.split()
    gen = torch.Generator().manual_seed(19)

    def halves(t):
        t = t.permute(*(axes.index(a) for a in "bths"), 4)
        return t[..., 0, :], t[..., 1, :], t[..., 2, :]

    buf = torch.randn([size[a] for a in axes] + [N], generator=gen).to(torch.bfloat16).to(dev)
    grad = torch.full_like(buf, 7.0)
    q, k, _ = halves(buf)
    gq, gk, gv = halves(grad)
    freq = torch.linspace(0.5, 0.01, N // 4, dtype=torch.float64, device=dev)
    dq, dk = grads_like(dev, 20, dict(q=q, k=k), fm)
    want = ss.qk_norm_rot_bwd(q.contiguous(), k.contiguous(), freq, dq, dk, feature_major=fm)
    got = ss.qk_norm_rot_bwd(q, k, freq, dq, dk, feature_major=fm, dq=gq, dk=gk)
    out, ref = ss.qk_norm_rot(q, k, freq, feature_major=fm), ss.qk_norm_rot(q.contiguous(), k.contiguous(), freq, feature_major=fm)
    torch.cuda.synchronize()
    assert torch.equal(gq, want["dq"]) and torch.equal(gk, want["dk"]) and (gv == 7).all()
    assert torch.equal(got["dwq"], want["dwq"]) and torch.equal(got["dwk"], want["dwk"])
    assert torch.equal(out[0], ref[0]) and torch.equal(out[1], ref[1])


@pytest.mark.parametrize("B,L,hq,hk,N,rot,fm", [(3, 20011, 1, 1, 16, 16, True), (1, 70001, 2, 1, 8, 4, True), (2, 333, 1, 2, 2, 2, True), (5, 1, 1, 1, 16, 16, True),
                                                (2, 4099, 8, 2, 64, 64, False), (1, 20011, 1, 1, 16, 16, False), (4, 2047, 20, 5, 80, 32, False), (3, 5003, 3, 1, 256, 128, False),
                                                (1, 9001, 2, 1, 33, 10, False), (7, 1, 4, 4, 40, 40, False)])
@pytest.mark.parametrize("io,interleaved", [("f32", False), ("bf16", True)])
def test_every_vector_counts_in_the_weights_gradient(ss, dev, B, L, hq, hk, N, rot, fm, io, interleaved):
    """Values of +-1 under an eps of 3 make every norm 2, positions of 0 turn nothing, and the gradients are odd whole numbers: each
    term of dw is +-1/2 or +-3/2, and each partial sum exact in fp32 (below 2^23).  So a single vector lost or doubled shows."""
    import torch
    gen = torch.Generator().manual_seed(N + L)
    dt = torch.float32 if io == "f32" else torch.bfloat16
    freq = torch.linspace(1.0, 0.1, rot // 2, dtype=torch.float64, device=dev)
    pos = torch.zeros(B, L, dtype=torch.int64, device=dev)
    w = torch.randn(N, generator=gen).to(dev)
    v = {s: (2 * torch.randint(0, 2, (B, L, h, N), generator=gen) - 1) for s, h in (("q", hq), ("k", hk))}
    d = {s: (2 * torch.randint(-2, 2, (B, L, h, N), generator=gen) + 1) for s, h in (("q", hq), ("k", hk))}
    up = {s: (t.permute(0, 2, 3, 1) if fm else t).to(dt).to(dev).contiguous() for s, t in d.items()}
    got = ss.qk_norm_rot_bwd(v["q"].to(dt).to(dev), v["k"].to(dt).to(dev), freq, up["q"], up["k"], wq=w, positions=pos, eps=3.0,
                             interleaved=interleaved, feature_major=fm)
    torch.cuda.synchronize()
    for s in "qk":
        assert 1.5 * B * L * max(hq, hk) < 1 << 23
        assert torch.equal(got["dw" + s].cpu().double() * 2, (v[s] * d[s]).sum((0, 1, 2)).double()), s


def test_c_names_of_the_binding(ss, dev):
    """The C entry points under their own names, with strides as three numbers: as the tensor calls."""
    import torch
    B, L, hq, hk, N, rot = 2, 33, 3, 1, 40, 32
    p = problem(dev, 21, B, L, hq, hk, N, rot, "bf16", 8, True)
    dq, dk = grads_like(dev, 22, p, False)
    q, k = ss.qk_norm_rot(**p, interleaved=True)
    want = ss.qk_norm_rot_bwd(dq_out=dq, dk_out=dk, **p, interleaved=True)
    new = {n: torch.empty_like(v) for n, v in dict(want, q=q, k=k).items()}
    ws = torch.empty(ss.ss_qk_norm_rot_bwd_workspace_bytes(B, L, hq, hk, N), dtype=torch.uint8, device=dev)
    s = torch.cuda.current_stream().cuda_stream
    head = (B, L, hq, hk, N, rot, ss.SS_BF16, ss.SS_QK_INTERLEAVED, EPS, p["q"].data_ptr(), p["q"].stride()[:3], p["k"].data_ptr(),
            p["k"].stride()[:3], *(p[n].data_ptr() for n in ("wq", "wk", "inv_freq", "positions")), 0)
    ss.ss_qk_norm_rot(*head, new["q"].data_ptr(), new["k"].data_ptr(), s)
    ss.ss_qk_norm_rot_bwd(*head, dq.data_ptr(), dk.data_ptr(), new["dq"].data_ptr(), new["dq"].stride()[:3], new["dk"].data_ptr(),
                          new["dk"].stride()[:3], new["dwq"].data_ptr(), new["dwk"].data_ptr(), ws.data_ptr(), ws.numel(), s)
    torch.cuda.synchronize()
    for n, v in dict(want, q=q, k=k).items():
        assert torch.equal(new[n], v), n
    with pytest.raises(ss.SsError):
        ss.ss_qk_norm_rot(*head[:5], 3, *head[6:], new["q"].data_ptr(), new["k"].data_ptr(), s)
