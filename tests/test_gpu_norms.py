"""The norms before and after a block on the GPU against 64 bits, and a block of them with the gated delta rule."""
import pytest
import torch

from blocks import BF16_REL, F32_REL, NORM_REL, close, gated64, gdr64, leaves, norm64, rel, residual64, silu64, up

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ss():
    import selective_state_space_62_amd as ss
    return ss


def rn(seed, *shape, io=F, scale=1.0, shift=0.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale + shift).to(io).cuda()


def sums_tol(rows):
    """fp32 sums of as many terms that do not all have one sign, relative to the sum's size: 2^-20 for the terms, and roundings of
    partial sums, of which no value passes more than rows / 1024 + 64."""
    return 2.0 ** -19 + (rows / 1024 + 64) * 2.0 ** -24


def near(name, got, want, tol, more):
    """Within tol of the result's norm and `more`, which the test derives."""
    off, size = float((got.detach().double().cpu() - want).norm()), float(want.norm())
    assert off <= tol * size + more, "%s: off by %.3g, %.3g allowed" % (name, off, tol * size + more)


SHAPES = [(1, 1, 1, 1), (2, 3, 2, 7), (3, 5, 1, 8), (1, 9, 4, 33), (2, 17, 5, 64), (4, 31, 3, 128), (1, 100, 2, 200), (2, 20, 1, 512), (1, 33, 2, 513),
          (1, 7, 1, 1000), (3, 3, 1, 1024), (2, 5, 1, 1025), (1, 11, 1, 2048), (1, 5, 1, 2560), (2, 3, 1, 5120), (1, 4, 1, 8191), (1, 3, 1, 8192),
          (1, 3000, 2, 16)]


@pytest.mark.parametrize("io", [F, BF])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("first,gate,weights", [(False, True, 1), (True, True, 1), (False, False, 1), (True, True, 2), (False, True, 0)])
def test_gated_norm(ss, shape, io, first, gate, weights):
    b, t, h, n = shape
    x, dy = rn(1, *shape, io=io), rn(3, *shape, io=io)
    z = rn(2, b, t, 5 + h * n, io=io)[..., 5:].unflatten(-1, (h, n)) if gate else None
    w = [None, rn(4, n, scale=0.3, shift=1.0), rn(4, h, n, scale=0.3, shift=1.0)][weights]
    lx, lz, lw = leaves(x, z, w if w is not None else torch.ones(n))
    want = gated64(lx, lz, lw, first)
    want.backward(up(dy))
    y = ss.gated_norm(x, z, w, gate_first=first)
    g = ss.gated_norm_bwd(x, z, dy, w, gate_first=first)
    tol = NORM_REL[io]
    close("y", y, want, tol)
    # the gradient of norm(a) is rho (p - a rho^2 mean(p a)), two terms of which the second is no larger than the first, rho |p|, each
    # within 2^-21 of itself (five roundings): their difference is within 2^-20 rho |p|, and what follows multiplies it
    ux, uz, uw, ud = up(x), up(z) if gate else None, up(w) if w is not None else torch.ones(n, dtype=torch.float64), up(dy)
    a = ux * silu64(uz) if first and gate else ux
    p = (ud * silu64(uz) if gate and not first else ud) * uw
    terms = p.norm(dim=-1, keepdim=True) / torch.sqrt((a * a).mean(-1, keepdim=True) + 1e-6)
    slope = (torch.sigmoid(uz) * (1 + uz * (1 - torch.sigmoid(uz)))) if gate else None
    near("dx", g["dx"], lx.grad, tol, 2.0 ** -20 * float((terms * (silu64(uz).abs().amax(-1, keepdim=True) if first and gate else 1.0)).norm()))
    if gate:
        near("dz", g["dz"], lz.grad, tol, 2.0 ** -20 * float((terms * (ux * slope).abs().amax(-1, keepdim=True)).norm()) if first else 0.0)
    else:
        assert g["dz"] is None
    close("dw", g["dw"], lw.grad, sums_tol(b * t * h))
    assert ss.gated_norm_bwd(x, z, dy, w, gate_first=first, need_dw=False)["dw"] is None


@pytest.mark.parametrize("first", [False, True])
def test_gated_norm_strides(ss, first):
    """x, z, dx and dz under strides of their own; other columns keep their values."""
    b, t, h, n = 2, 9, 3, 40
    rows = rn(5, b, t, 400, io=BF)
    x, z = rows[..., 3:123].unflatten(-1, (h, n)), rows[..., 123:243].unflatten(-1, (h, n))
    dy, w = rn(6, b, t, h, n, io=BF), rn(7, n)
    out = torch.full((t, b, 400), 9.0, dtype=BF, device="cuda")
    dx = out[..., 1:121].unflatten(-1, (h, n)).transpose(0, 1)
    dz = torch.empty(b, h, t, n, dtype=BF, device="cuda").transpose(1, 2)
    g = ss.gated_norm_bwd(x, z, dy, w, gate_first=first, dx=dx, dz=dz)
    ref = ss.gated_norm_bwd(x.contiguous(), z.contiguous(), dy, w, gate_first=first)
    assert torch.equal(g["dx"], ref["dx"]) and torch.equal(g["dz"], ref["dz"]) and torch.equal(g["dw"], ref["dw"])
    assert bool((out[..., 0] == 9).all()) and bool((out[..., 121:] == 9).all())
    assert torch.equal(ss.gated_norm(x, z, w, gate_first=first), ss.gated_norm(x.contiguous(), z.contiguous(), w, gate_first=first))


def test_gated_norm_shapes(ss):
    x, z, w = rn(1, 6, 32), rn(2, 6, 32), rn(3, 32)
    y = ss.gated_norm(x, z, w)
    assert y.shape == (6, 32)
    assert torch.equal(ss.gated_norm(x.view(2, 3, 32), z.view(2, 3, 32), w).view(6, 32), y)
    assert ss.gated_norm(torch.empty(2, 0, 4, device="cuda")).shape == (2, 0, 4)
    g = ss.gated_norm_bwd(torch.empty(2, 0, 4, device="cuda"), None, torch.empty(2, 0, 4, device="cuda"))
    assert float(g["dw"].abs().max()) == 0.0 and g["dw"].shape == (4,)


def test_gated_norm_special_values(ss):
    """Gates that are closed, wide open or infinite; rows of zeros; NaN in a row stays there."""
    x, w = rn(1, 1, 8, 1, 64), rn(2, 64)
    z = torch.zeros(1, 8, 1, 64, device="cuda")
    z[0, 0], z[0, 1], z[0, 2] = -200.0, 200.0, -80.0
    x[0, 3] = 0.0
    x[0, 4, 0, 5] = float("nan")
    y = ss.gated_norm(x, z, w)
    assert float(y[0, 0].abs().max()) == 0.0 and float(y[0, 3].abs().max()) == 0.0
    assert bool(torch.isnan(y[0, 4]).all()) and bool(torch.isfinite(y[0, [0, 1, 2, 3, 5, 6, 7]]).all())
    close("open", y[0, 1], gated64(up(x), up(z), up(w), False)[0, 1], NORM_REL[F])
    g = ss.gated_norm_bwd(x, z, torch.ones_like(x), w, need_dw=False)
    assert bool(torch.isfinite(g["dx"][0, [0, 1, 2, 3, 5]]).all()) and bool(torch.isfinite(g["dz"][0, [0, 1, 2, 3, 5]]).all())


@pytest.mark.parametrize("io,rio", [(F, F), (BF, F), (BF, BF)])
@pytest.mark.parametrize("rows,n", [(1, 1), (3, 5), (2, 8), (7, 64), (33, 333), (5, 768), (4, 1000), (1025, 48), (9, 2560), (2, 4097), (3, 8192)])
@pytest.mark.parametrize("post,scaled,res", [(True, True, True), (False, False, True), (True, False, True), (False, True, False)])
def test_residual_norm(ss, io, rio, rows, n, post, scaled, res):
    x, r0 = rn(1, rows, n, io=io), rn(2, rows, n, io=rio, scale=3.0) if res else None
    w, wp = rn(3, n, scale=0.2, shift=1.0), rn(4, n, scale=0.2, shift=1.0) if post else None
    sc = rn(5, n, scale=0.2, shift=0.5) if scaled else None
    dy, dr = rn(6, rows, n, io=io), rn(7, rows, n, io=rio)
    kw = dict(w_post=wp, post=post, scale=sc, alpha=0.7)
    y, r = ss.residual_norm(x, r0, w, residual_dtype=rio, **kw)
    assert r.dtype == rio and y.dtype == io
    g = ss.residual_norm_bwd(x, r, dy, dr, w, **kw)
    lx, lr, lw, lwp, lsc = leaves(x, r0, w, wp, sc)
    wy, wr = residual64(lx, lr, lw, lwp, post, lsc, 0.7, rounded=up(r))
    ((wy * up(dy)).sum() + (wr * up(dr)).sum()).backward()
    close("r", r, wr, NORM_REL[rio])
    close("y", y, wy, NORM_REL[io])
    # a norm's gradient is within 2^-20 rho |p| (see test_gated_norm); an error of dr passes on times what dr is multiplied by
    ur, ux, ud = up(r), up(x), up(dy)
    by = 0.7 * (up(sc) if scaled else torch.ones(n, dtype=torch.float64))
    rho = 1 / torch.sqrt((ur * ur).mean(-1, keepdim=True) + 1e-6)
    off_r = 2.0 ** -20 * (rho * (ud * up(w)).norm(dim=-1, keepdim=True))             # of each row of dr
    m = norm64(ux, up(wp)) if post else ux
    if res:
        near("dres", g["dres"], lr.grad, NORM_REL[rio], float(off_r.norm()))
        dr_all = lr.grad
    else:
        dr_all = up(g["dres"])
    reach = by.abs().max()
    off_x = off_r * reach
    if post:
        rho_x = 1 / torch.sqrt((ux * ux).mean(-1, keepdim=True) + 1e-6)
        off_x = 2 * rho_x * up(wp).abs().max() * off_x + 2.0 ** -20 * rho_x * (dr_all * by * up(wp)).norm(dim=-1, keepdim=True)
    near("dx", g["dx"], lx.grad, NORM_REL[io], float(off_x.norm()))
    for name, l, f in (("dw", lw, None), ("dw_post", lwp, by * norm64(ux)), ("dscale", lsc, 0.7 * m)):
        if l is None:
            assert g[name] is None
        else:
            more = 0.0 if f is None else float((off_r * f.abs().amax(-1, keepdim=True)).sum())
            near(name, g[name], l.grad, sums_tol(rows), more)


def test_residual_norm_in_place(ss):
    """res_out may be res and dres the gradient of r itself; without a gradient of r it counts as zero."""
    x, r0, w, dy, dr = rn(1, 50, 768, io=BF), rn(2, 50, 768), rn(3, 768), rn(4, 50, 768, io=BF), rn(5, 50, 768)
    y, r = ss.residual_norm(x, r0, w)
    mine = r0.clone()
    y2, r2 = ss.residual_norm(x, mine, w, res_out=mine)
    assert r2 is mine and torch.equal(y, y2) and torch.equal(r, mine)
    g = ss.residual_norm_bwd(x, r, dy, dr, w)
    kept = dr.clone()
    g2 = ss.residual_norm_bwd(x, r, dy, kept, w, dres=kept)
    assert torch.equal(g["dres"], kept) and torch.equal(g["dx"], g2["dx"])
    none, zero = ss.residual_norm_bwd(x, r, dy, None, w), ss.residual_norm_bwd(x, r, dy, torch.zeros_like(dr), w)
    assert torch.equal(none["dx"], zero["dx"])
    empty = ss.residual_norm_bwd(x[:0], r[:0], dy[:0], None, w)
    assert float(empty["dw"].abs().max()) == 0.0


def test_many_rows_are_all_counted(ss):
    """Weights' gradients of terms that fp32 adds exactly, whatever the order: none is lost."""
    rows, n = 40_003, 24
    x = torch.ones(rows, 1, 1, n, device="cuda")
    dy = torch.randint(-8, 9, (rows, 1, 1, n), generator=torch.Generator().manual_seed(1)).float().cuda()
    eps = 3.0                                              # x / sqrt(1 + 3) is 1/2 exactly
    g = ss.gated_norm_bwd(x, None, dy, eps=eps)
    assert torch.equal(g["dw"], dy.sum((0, 1, 2)) / 2)
    r = ss.residual_norm_bwd(x.view(rows, n), x.view(rows, n), dy.view(rows, n), None, eps=eps)
    assert torch.equal(r["dw"], dy.view(rows, n).sum(0) / 2)
    heads = ss.gated_norm_bwd(x.view(rows // 7, 7, 1, n).expand(rows // 7, 7, 1, n), None, dy.view(rows // 7, 7, 1, n).contiguous(),
                              torch.ones(1, n, device="cuda"), eps=eps) if rows % 7 == 0 else None
    assert heads is None or torch.equal(heads["dw"][0], dy.sum((0, 1, 2)) / 2)


def test_norms_repeat_and_replay(ss):
    x, z, w, dy = rn(1, 4, 100, 8, 128, io=BF), rn(2, 4, 100, 8, 128, io=BF), rn(3, 128), rn(4, 4, 100, 8, 128, io=BF)
    res, wr = rn(5, 400, 1024), rn(6, 1024)
    graph = torch.cuda.CUDAGraph()
    run = lambda: (ss.gated_norm(x, z, w), *ss.gated_norm_bwd(x, z, dy, w).values(), *ss.residual_norm(x.view(400, 1024), res, wr),  # noqa: E731
                   *[v for v in ss.residual_norm_bwd(x.view(400, 1024), res, dy.view(400, 1024), None, wr).values() if v is not None])
    run()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        captured = run()
    for k in range(3):
        x.copy_((x.float() * 0.5 + 0.1 * k).to(BF))
        graph.replay()
        eager = run()
        again = run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, eager)) and all(torch.equal(a, b) for a, b in zip(again, eager))


@pytest.mark.parametrize("call,error", [
    (lambda ss, x: ss.gated_norm(x.double()), TypeError), (lambda ss, x: ss.gated_norm(x.cpu()), ValueError),
    (lambda ss, x: ss.gated_norm(x, x[:, :3]), ValueError), (lambda ss, x: ss.gated_norm(x, None, torch.ones(5, device="cuda")), ValueError),
    (lambda ss, x: ss.gated_norm(x, eps=0.0), Exception), (lambda ss, x: ss.gated_norm(x.transpose(-1, -2)), ValueError),
    (lambda ss, x: ss.gated_norm(x, y=x), Exception), (lambda ss, x: ss.gated_norm_bwd(x, None, x, dz=x), ValueError),
    (lambda ss, x: ss.gated_norm_bwd(x, None, None), ValueError), (lambda ss, x: ss.residual_norm(x, x.bfloat16()), TypeError),
    (lambda ss, x: ss.residual_norm(x.transpose(0, 1)), ValueError), (lambda ss, x: ss.residual_norm(x, w_post=x[0, 0]), ValueError),
    (lambda ss, x: ss.residual_norm_bwd(x, None, x), ValueError), (lambda ss, x: ss.residual_norm_bwd(x, x, x[:1]), ValueError),
    (lambda ss, x: ss.gated_norm(torch.zeros(1, 9000, device="cuda")), Exception),
])
def test_refusals(ss, call, error):
    with pytest.raises(error):
        call(ss, rn(1, 4, 6, 32))


@pytest.mark.parametrize("io", [F, BF])
def test_a_block(ss, io):
    """What a recurrent layer runs between its products: norm and rotation of queries and keys, the gated delta rule, the gated norm of
    its heads, the residual norm; forward, and its gradients, against 64 bits."""
    B, L, hk, hv, dk, dv = 2, 100, 2, 4, 32, 48
    N = hv * dv
    rows = rn(1, B, L, 2 * hk * dk + 2 * N, io=io)         # a projection's rows: q, k, v, z
    q, k = rows[..., :hk * dk].unflatten(-1, (hk, dk)), rows[..., hk * dk:2 * hk * dk].unflatten(-1, (hk, dk))
    v, z = rows[..., 2 * hk * dk:2 * hk * dk + N].unflatten(-1, (hv, dv)), rows[..., 2 * hk * dk + N:].unflatten(-1, (hv, dv))
    unit = torch.full((dk,), dk ** -0.5, device="cuda")
    g, beta = -0.2 * torch.rand(B, L, hv, generator=torch.Generator().manual_seed(2)).cuda(), torch.sigmoid(rn(3, B, L, hv))
    res, wn, w = rn(4, B, L, N), rn(5, dv, scale=0.1, shift=1.0), rn(6, N, scale=0.1, shift=1.0)
    dy, dr = rn(7, B, L, N, io=io), rn(8, B, L, N)
    freq = 100.0 ** (-torch.arange(dk // 2, dtype=torch.float64, device="cuda") / (dk // 2))

    qn, kn = ss.qk_norm_rot(q, k, freq, unit, unit)
    o, _ = ss.gdr_fwd(qn, kn, v, g, beta)
    n = ss.gated_norm(o, z, wn)
    y, r = ss.residual_norm(n.view(B, L, N), res, w)
    gr = ss.residual_norm_bwd(n.view(B, L, N), r, dy, dr, w)
    gn = ss.gated_norm_bwd(o, z, gr["dx"].view(B, L, hv, dv), wn)
    gd = ss.gdr_bwd(qn, kn, v, g, beta, gn["dx"])
    gq = ss.qk_norm_rot_bwd(q, k, freq, gd["dq"], gd["dk"], unit, unit)

    lrow, lg, lb, lres, lwn, lw = leaves(rows, g, beta, res, wn, w)
    lq, lk = lrow[..., :hk * dk].unflatten(-1, (hk, dk)), lrow[..., hk * dk:2 * hk * dk].unflatten(-1, (hk, dk))
    lv, lz = lrow[..., 2 * hk * dk:2 * hk * dk + N].unflatten(-1, (hv, dv)), lrow[..., 2 * hk * dk + N:].unflatten(-1, (hv, dv))
    ang = torch.arange(L, dtype=torch.float64)[:, None, None] * up(freq)

    def turn(x):
        a = norm64(x, up(unit))
        a1, a2 = a[..., :dk // 2], a[..., dk // 2:]
        return torch.cat((a1 * ang.cos() - a2 * ang.sin(), a2 * ang.cos() + a1 * ang.sin()), -1)
    wo, _ = gdr64(turn(lq), turn(lk), lv, lg, lb, None, dk ** -0.5)
    wy, wr = residual64((norm64(wo, lwn) * silu64(lz)).flatten(-2), lres, lw, None, False, None, 1.0)
    ((wy * up(dy)).sum() + (wr * up(dr)).sum()).backward()
    # up to seven results in a row are rounded to the I/O type: each adds its half step at most
    tol = 7 * 2.0 ** -8 if io == BF else 4 * F32_REL
    close("y", y, wy, tol)
    close("r", r, wr, tol)
    close("dres", gr["dres"], lres.grad, tol)
    close("dw", gr["dw"], lw.grad, tol)
    close("dwn", gn["dw"], lwn.grad, tol)
    close("dz", gn["dz"], lrow.grad[..., 2 * hk * dk + N:].unflatten(-1, (hv, dv)), tol)
    close("dv", gd["dv"], lrow.grad[..., 2 * hk * dk:2 * hk * dk + N].unflatten(-1, (hv, dv)), tol)
    close("dq", gq["dq"], lrow.grad[..., :hk * dk].unflatten(-1, (hk, dk)), tol)
    close("dk", gq["dk"], lrow.grad[..., hk * dk:2 * hk * dk].unflatten(-1, (hk, dk)), tol)
    close("dbeta", gd["dbeta"], lb.grad, tol)
    assert rel(gd["dg"], lg.grad) <= 4 * tol
