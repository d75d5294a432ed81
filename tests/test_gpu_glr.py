"""The gated linear recurrence on the GPU against the formulas in 64 bits."""
import numpy as np
import pytest

import bounds
from bounds import U, V, check, recur, sigmoid
from gpu_util import log, to_f64

pytestmark = pytest.mark.gpu
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
SCALE = 8.0


@pytest.fixture(scope="module")
def dev():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return torch.device("cuda:0")


@pytest.fixture(scope="module")
def ss():
    import selective_state_space_62_amd as m
    return m


def problem(dev, seed, batch, dim, L, io="bf16", kind="normalised", i=True, z=True, h0=True, decay=True, bias=True,
            step=False):
    """Seeded inputs on the GPU, every value exact in its type."""
    import torch
    gen = torch.Generator().manual_seed(seed)
    dt = torch.float32 if io == "f32" else torch.bfloat16
    full = (batch, dim) if step else (batch, dim, L)

    def n(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=gen).to(dtype).to(dev)

    p = dict(x=n(*full, dtype=dt), r=n(*full, dtype=dt), i=n(*full, dtype=dt) if i else None,
             z=n(*full, dtype=dt) if z else None, kind=kind)
    if kind == "convex":
        p["decay"] = torch.rand(dim, generator=gen).to(dev) if decay else None
    else:   # from fast decays to ones within 1e-3 of 1, where 1 - a^2 cancels
        p["decay"] = (torch.rand(dim, generator=gen) * 10 - 9).to(dev)
    p["r_bias"] = n(dim) if bias else None
    p["i_bias"] = n(dim) if bias and i else None
    p["h0"] = n(batch, dim) if h0 else None
    return p


def f64(t):
    return None if t is None else to_f64(t)


def forward(p, adds):
    """Gates, states and outputs with their bounds (batch, D, L)."""
    col = lambda t: V(0.0) if t is None else V(f64(t)[:, None])  # noqa: E731
    x, r = V(f64(p["x"])), V(f64(p["r"])) + col(p["r_bias"])
    s, oms = sigmoid(r), sigmoid(-r)
    g = {"s": s, "oms": oms, "x": x}
    if p["kind"] == "convex":
        f = col(p["decay"])
        one = V(1.0) - f
        g["a"], g["m"], g["one"] = f + one * s, one * oms, one
    else:
        d = f64(p["decay"])[:, None]
        soft = np.logaddexp(0.0, d)
        # softplus from log2(1 + e^-|d|): the exponent's rounding, exp2, the sum, log2 and the last sum
        l = V(SCALE * soft, SCALE * soft * U * (2 * np.abs(d) + 10))
        ls = l * s
        a = np.exp(-ls.v)
        g["a"] = V(a, a * (ls.e + 2 * U * np.abs(ls.v) + 2 * U))
        q = -np.expm1(-2 * ls.v)
        # by the polynomial below w = 1/8 (terms: 6 roundings and 4.3e-8 dropped), else 1 - a^2
        rel = np.where(2 * ls.v < 0.125, (ls.e / np.maximum(ls.v, 1e-300)) + 8 * U, (2 * a * g["a"].e + 2 * U) / np.maximum(q, 0.1))
        g["rel_q"], g["ls"] = rel, ls
        g["m"] = V(np.sqrt(q), np.sqrt(q) * (0.5 * rel + 4 * U))
        k = ls.v / np.maximum(np.sqrt(q), 1e-300)
        g["k"] = V(k, k * (ls.e / np.maximum(ls.v, 1e-300) + 0.5 * rel + 4 * U))
    g["ix"] = x
    if p["i"] is not None:
        i = V(f64(p["i"])) + col(p["i_bias"])
        g["iota"], g["omi"] = sigmoid(i), sigmoid(-i)
        g["ix"] = x * g["iota"]
    h0 = np.zeros(x.v.shape[:2]) if p["h0"] is None else f64(p["h0"])
    g["u"] = g["m"] * g["ix"]
    g["h"], g["before"] = recur(g["a"], g["u"], V(h0), adds)
    z = None if p["z"] is None else V(f64(p["z"]))
    g["y"] = g["h"] if z is None else g["h"] * bounds.silu(z)
    return g


def backward(p, g, dy, dh, adds):
    dy = V(dy)
    w = dy if p["z"] is None else dy * bounds.silu(V(f64(p["z"])))
    # G_t = a_t (w_t + G_(t+1)): the recurrence from the end over a and a w
    G, after = recur(g["a"][..., ::-1], (g["a"] * w)[..., ::-1], V(dh), adds)
    gg = w + after[..., ::-1]
    out = {"dh0": G[..., -1]}
    if p["kind"] == "convex":
        da = gg * (g["before"] - g["ix"])
        out["dr"] = da * g["m"] * g["s"]
        dd, factor = da * g["oms"], 1.0
    else:
        dd = gg * g["a"] * (g["a"] * g["k"] * g["ix"] - g["ls"] * g["before"])
        out["dr"] = dd * g["oms"]
        d = f64(p["decay"])
        factor = 1.0 / (1.0 + np.exp(-d)) / np.logaddexp(0.0, d)
    gm = gg * g["m"]
    out["dx"] = gm
    if p["i"] is not None:
        out["dx"] = gm * g["iota"]
        out["di"] = gm * g["ix"] * g["omi"]
    if p["z"] is not None:
        z = V(f64(p["z"]))
        out["dz"] = dy * g["h"] * (sigmoid(z) * (V(1.0) + z * sigmoid(-z)))
    batch, _, L = dy.v.shape
    steps = L / 64 + batch + 24
    for name, per in (("ddecay", dd), ("dr_bias", out["dr"]), ("di_bias", out.get("di"))):
        if per is not None:
            s = per.sum((0, 2), steps)
            f = factor if name == "ddecay" else 1.0
            out[name] = V(s.v * f, np.abs(s.e * f) + 30 * U * np.abs(s.v * f))
    return out


def adds(L):
    """Roundings between a token's term and the row's end besides the ones counted per token: 8 within a
    lane, 7 over the wave, 4 over its waves, twice for the replay, one for each tile."""
    return 40 + L / 512


def run_fwd(ss, p, **kw):
    import torch
    y, h = ss.glr_fwd(**p, **kw)
    torch.cuda.synchronize()
    return y, h


FORMS = [("convex", "f32", True, True, True), ("convex", "bf16", False, False, False), ("normalised", "f32", True, False, True),
         ("normalised", "bf16", True, True, True), ("normalised", "f32", False, True, False), ("convex", "bf16", True, False, True)]
# one token, odd ones, the borders of a lane (8), of 16 lanes (128), a wave (512), two and four waves (1024, 2048), and past them
LENGTHS = [1, 2, 7, 8, 9, 63, 127, 128, 129, 511, 512, 513, 1023, 1025, 2047, 2048, 2049, 4100, 6145, 8193, 10247]


@pytest.mark.parametrize("kind,io,i,z,h0", FORMS)
@pytest.mark.parametrize("L", LENGTHS)
def test_forward(ss, dev, L, kind, io, i, z, h0):
    p = problem(dev, 100 + L, 2, 5, L, io, kind, i, z, h0)
    y, h = run_fwd(ss, p)
    g = forward(p, adds(L))
    check("y", f64(y), g["y"], HALF[io])
    check("h_final", f64(h), g["h"][..., -1], 0.0)


@pytest.mark.parametrize("kind,io,i,z,h0", FORMS)
@pytest.mark.parametrize("L", LENGTHS)
def test_backward(ss, dev, L, kind, io, i, z, h0):
    import torch
    p = problem(dev, 200 + L, 2, 5, L, io, kind, i, z, h0)
    gen = torch.Generator().manual_seed(L)
    dy = torch.randn(p["x"].shape, generator=gen).to(p["x"].dtype).to(dev)
    dh = torch.randn((2, 5), generator=gen).to(dev)
    want = backward(p, forward(p, adds(L)), f64(dy), f64(dh), adds(L))
    ckpt = torch.full((ss.glr_ckpt_numel(2, 5, L),), float("nan"), device=dev)
    ss.glr_fwd(**p, ckpt=ckpt)
    for stored in (None, ckpt):
        got = ss.glr_bwd(dy=dy, dh_final=dh, ckpt=stored, **p)
        torch.cuda.synchronize()
        for name, v in want.items():
            check(name + (" from stored states" if stored is not None else ""), f64(got[name]), v,
                  HALF[io] if got[name].dtype == torch.bfloat16 else 0.0)
        for name in set(got) - set(want):
            assert got[name] is None, name


@pytest.mark.parametrize("kind", ["convex", "normalised"])
@pytest.mark.parametrize("batch,dim,L", [(3, 700, 5), (1, 2100, 300), (2, 513, 2500), (1, 256, 16391)])
def test_many_rows(ss, dev, kind, batch, dim, L):
    """Enough rows for the plan that gives each of them to one workgroup."""
    import torch
    p = problem(dev, 300 + L, batch, dim, L, "bf16", kind)
    y, h = run_fwd(ss, p)
    g = forward(p, adds(L))
    check("y", f64(y), g["y"], HALF["bf16"])
    check("h_final", f64(h), g["h"][..., -1], 0.0)
    dy = torch.randn(p["x"].shape, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(dev)
    got = ss.glr_bwd(dy=dy, **p)
    torch.cuda.synchronize()
    for name, v in backward(p, g, f64(dy), np.zeros((batch, dim)), adds(L)).items():
        check(name, f64(got[name]), v, HALF["bf16"] if got[name].dtype == torch.bfloat16 else 0.0)


@pytest.mark.parametrize("kind,io", [("convex", "f32"), ("normalised", "bf16")])
def test_long_rows(ss, dev, kind, io):
    """Tens of thousands of tokens in few rows: more tiles than are joined from one state."""
    import torch
    L = 2048 * 67 + 5
    p = problem(dev, 21, 1, 3, L, io, kind)
    y, h = run_fwd(ss, p)
    g = forward(p, adds(L))
    check("y", f64(y), g["y"], HALF[io])
    check("h_final", f64(h), g["h"][..., -1], 0.0)
    dy = torch.randn(p["x"].shape, generator=torch.Generator().manual_seed(1)).to(p["x"].dtype).to(dev)
    dh = torch.ones(1, 3, device=dev)
    want = backward(p, g, f64(dy), f64(dh), adds(L))
    ckpt = torch.full((ss.glr_ckpt_numel(1, 3, L),), float("nan"), device=dev)
    ss.glr_fwd(**p, ckpt=ckpt)
    for stored in (None, ckpt):
        got = ss.glr_bwd(dy=dy, dh_final=dh, ckpt=stored, **p)
        torch.cuda.synchronize()
        for name, v in want.items():
            check(name, f64(got[name]), v, HALF[io] if got[name].dtype == torch.bfloat16 else 0.0)


@pytest.mark.parametrize("pieces,extra,kind,io", [(64, 1, "convex", "bf16"), (127, 0, "normalised", "f32"), (128, 9, "normalised", "bf16"),
                                                  (131, -3, "convex", "f32"), (132, 0, "normalised", "bf16")])
def test_split_rows_of_several_pieces(ss, dev, pieces, extra, kind, io):
    """Rows split into tiles of two and four times 2048 tokens, the last tile whole or missing some of its pieces; states stored
    every 2048 tokens."""
    import torch
    L = 2048 * pieces + extra
    p = problem(dev, 28, 2, 1, L, io, kind)
    ckpt = torch.full((ss.glr_ckpt_numel(2, 1, L),), float("nan"), device=dev)
    y, h = run_fwd(ss, p, ckpt=ckpt)
    g = forward(p, adds(L))
    check("y", f64(y), g["y"], HALF[io])
    check("h_final", f64(h), g["h"][..., -1], 0.0)
    states = ckpt.view(2, 1, -1)
    assert torch.equal(states[..., 0], p["h0"])
    check("ckpt", f64(states[..., 1:]), g["h"][..., 2047:L - 1:2048], 0.0)


def test_sixteen_waves_to_a_row(ss, dev):
    """bf16 rows of 2^17 tokens, enough of them to have a workgroup each: like the split of the same rows, up to the
    rounding of y (half a step each) and of the states' joining (within 1e-4 of a row's largest, as the bounds above)."""
    import torch
    rows, L = 260, (1 << 17) + 3
    p = problem(dev, 23, 1, rows, L, "bf16", "convex", z=False)
    ckpt = torch.full((ss.glr_ckpt_numel(1, rows, L),), float("nan"), device=dev)
    y, h = ss.glr_fwd(**p, ckpt=ckpt)
    dy = torch.randn_like(p["x"])
    g = ss.glr_bwd(dy=dy, ckpt=ckpt, **p)
    few = {k: v[:, :9].contiguous() if torch.is_tensor(v) and v.dim() > 1 else v[:9].contiguous() if torch.is_tensor(v) else v
           for k, v in p.items()}
    y9, h9 = ss.glr_fwd(**few)
    g9 = ss.glr_bwd(dy=dy[:, :9].contiguous(), **few)
    torch.cuda.synchronize()
    for name, a, b in [("y", y, y9), ("h", h, h9)] + [(k, g[k], g9[k]) for k in ("dx", "dr", "di", "dh0")]:
        a, b = a[:, :9].float(), b.float()
        top = b.abs().amax(-1, keepdim=True) if b.dim() == 3 else b.abs().max()
        assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 1e-4 * top).all(), name
    for name in ("ddecay", "dr_bias", "di_bias"):
        assert float((g[name][:9] - g9[name]).abs().max()) <= 1e-4 * float(g9[name].abs().max()) + 1e-2, name


@pytest.mark.parametrize("rows,L,kind,io", [(319, 32771, "normalised", "bf16"), (257, 40000, "convex", "f32"), (330, (1 << 17) + 3, "convex", "bf16"),
                                            (320, 32771, "normalised", "bf16"), (320, 33000, "convex", "f32")])
def test_about_as_many_long_rows_as_compute_units(ss, dev, rows, L, kind, io):
    """Rows on both sides of the border between a workgroup to each and the split: like the split of the last nine of them, up to
    the rounding of y (half a step each) and of the states' joining (within 1e-4 of a row's largest, as the bounds above)."""
    import torch
    p = problem(dev, 29, 1, rows, L, io, kind, z=False)
    ckpt = torch.full((ss.glr_ckpt_numel(1, rows, L),), float("nan"), device=dev)
    y, h = ss.glr_fwd(**p, ckpt=ckpt)
    dy = torch.randn_like(p["x"])
    g = ss.glr_bwd(dy=dy, **p)
    stored = ss.glr_bwd(dy=dy, ckpt=ckpt, **p)
    few = {k: v[:, -9:].contiguous() if torch.is_tensor(v) and v.dim() > 1 else v[-9:].contiguous() if torch.is_tensor(v) else v
           for k, v in p.items()}
    y9, h9 = ss.glr_fwd(**few)
    g9 = ss.glr_bwd(dy=dy[:, -9:].contiguous(), **few)
    torch.cuda.synchronize()
    for k in ("dx", "dr", "di", "dh0", "ddecay", "dr_bias", "di_bias"):
        assert torch.equal(g[k], stored[k]), k
    for name, a, b in [("y", y, y9), ("h", h, h9)] + [(k, g[k], g9[k]) for k in ("dx", "dr", "di", "dh0")]:
        a, b = a[:, -9:].float(), b.float()
        top = b.abs().amax(-1, keepdim=True) if b.dim() == 3 else b.abs().max()
        assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 1e-4 * top).all(), name
    for name in ("ddecay", "dr_bias", "di_bias"):
        assert float((g[name][-9:] - g9[name]).abs().max()) <= 1e-4 * float(g9[name].abs().max()) + 1e-2, name


def test_zero_decays_join_across_tiles(ss, dev):
    """Floors of 0 and closed gates make maps of all zeros, which still are maps."""
    import torch
    L = 5 * 2048
    p = problem(dev, 22, 1, 4, L, "f32", "convex", z=False)
    p["decay"].zero_()
    p["r"][:, :, 2048:4096] = float("-inf")     # a = 0 throughout a tile
    p["x"][:, 0, 2048:4096] = 0                 # and nothing enters
    y, h = run_fwd(ss, p)
    assert not y[0, 0, 2048:4096].any()
    own = {k: v[:, :, 4096:] if k in ("x", "r", "i") else v for k, v in p.items()}
    own["h0"] = y[:, :, 4095].contiguous()
    g = forward(own, adds(L))
    check("y", f64(y[:, :, 4096:]), g["y"], HALF["f32"])
    gr = ss.glr_bwd(dy=torch.ones_like(y), **p)
    torch.cuda.synchronize()
    assert all(torch.isfinite(v).all() for v in gr.values() if v is not None)
    assert not gr["dh0"].isnan().any()


def test_gradients_against_differences(ss, dev):
    """The formulas' gradients, which the kernels are held to above, against central differences of the 64-bit forward."""
    rng = np.random.default_rng(5)
    B, D, L, eps = 2, 3, 6, 1e-6
    for kind in ("convex", "normalised"):
        import torch
        base = {k: rng.standard_normal((B, D, L)) for k in ("x", "r", "i", "z")}
        base["decay"] = rng.uniform(0.1, 0.9, D) if kind == "convex" else rng.uniform(-4, 1, D)
        base["r_bias"], base["i_bias"], base["h0"] = rng.standard_normal(D), rng.standard_normal(D), rng.standard_normal((B, D))
        dy, dh = rng.standard_normal((B, D, L)), rng.standard_normal((B, D))
        as_t = lambda d: {k: torch.from_numpy(v) for k, v in d.items()}  # noqa: E731

        def loss(d):
            g = forward64(dict(as_t(d), kind=kind))
            return float((g["y"].v * dy).sum() + (g["h"].v[..., -1] * dh).sum())

        p = dict(as_t(base), kind=kind)
        want = backward64(p, dy, dh)
        for name, grad in (("x", "dx"), ("r", "dr"), ("i", "di"), ("z", "dz"), ("decay", "ddecay"), ("r_bias", "dr_bias"),
                           ("i_bias", "di_bias"), ("h0", "dh0")):
            num = np.empty_like(base[name])
            for at in np.ndindex(num.shape):
                up, dn = {k: v.copy() for k, v in base.items()}, {k: v.copy() for k, v in base.items()}
                up[name][at] += eps
                dn[name][at] -= eps
                num[at] = (loss(up) - loss(dn)) / (2 * eps)
            # differences of values near 10 with 1e-16 of them over 2e-6, and eps^2 of a third derivative
            assert np.max(np.abs(num - want[grad].v)) < 1e-7, (kind, name)


def _double(t):
    return None if t is None else t.double().numpy() if hasattr(t, "double") else t


def forward64(p):
    global f64
    keep, f64 = f64, _double
    try:
        return forward(p, 0)
    finally:
        f64 = keep


def backward64(p, dy, dh):
    global f64
    keep, f64 = f64, _double
    try:
        return backward(p, forward(p, 0), dy, dh, 0)
    finally:
        f64 = keep


@pytest.mark.parametrize("kind", ["convex", "normalised"])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("i,z", [(True, True), (False, False)])
@pytest.mark.parametrize("batch,dim", [(1, 1), (3, 37), (5, 1030)])
def test_step_is_one_token_of_the_sequence(ss, dev, kind, io, i, z, batch, dim):
    import torch
    T = 4
    p = problem(dev, 7, batch, dim, T, io, kind, i, z)
    g = forward(p, adds(T))
    state = p["h0"].clone()
    for t in range(T):
        tok = {k: None if p[k] is None else p[k][..., t].contiguous() for k in ("x", "r", "i", "z")}
        vec = {k: p[k] for k in ("decay", "r_bias", "i_bias", "kind")}
        other = torch.empty_like(state)
        y2 = ss.glr_step(state, **tok, **vec, state_out=other)
        kept = state.clone()
        y = ss.glr_step(state, **tok, **vec)
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(state, other) and not torch.equal(kept, state)
        check("y %d" % t, f64(y), g["y"][..., t], HALF[io])
    check("state", f64(state), g["h"][..., -1], 0.0)


@pytest.mark.parametrize("kind,closed", [("convex", float("inf")), ("normalised", float("-inf"))])
@pytest.mark.parametrize("L", [40, 3000])
def test_padding_tokens_leave_the_state_alone(ss, dev, kind, closed, L):
    """Rows padded behind, before and altogether: the state of the tokens that are there (exactly that of none), zero
    gradients of the others, finite everywhere."""
    import torch
    p = problem(dev, 11, 3, 6, L, "f32", kind, z=False)
    n = L - 13
    p["r"][0, :, n:] = closed
    p["r"][1, :, :n] = closed
    p["r"][2] = closed
    y, h = run_fwd(ss, p)
    own = {k: v[:1, :, :n] if k in ("x", "r", "i") else v[:1] if k == "h0" else v for k, v in p.items()}
    end = forward(own, adds(L))["h"][..., -1]
    for name, v in (("y of the last token", y[:1, :, n - 1]), ("y of the last padding", y[:1, :, -1]), ("h_final", h[:1])):
        check(name, f64(v), end, 0.0)
    assert torch.equal(y[1, :, 0], p["h0"][1]) and torch.equal(y[1, :, n - 1], p["h0"][1])
    assert torch.equal(h[2], p["h0"][2]) and torch.equal(y[2], p["h0"][2][:, None].expand(-1, L))
    dy = torch.ones_like(y)
    g = ss.glr_bwd(dy=dy, **p)
    torch.cuda.synchronize()
    for name in ("dx", "dr", "di"):
        assert torch.isfinite(g[name]).all(), name
        assert not g[name][0, :, n:].any() and not g[name][1, :, :n].any() and not g[name][2].any(), name
    assert torch.equal(g["dh0"][2], torch.full_like(g["dh0"][2], float(L)))
    for name in ("ddecay", "dr_bias", "di_bias"):
        assert torch.isfinite(g[name]).all(), name


def test_extreme_gates_and_decays(ss, dev):
    """Gates of +-100, floors of 0 and 1, decays whose softplus underflows or is large: finite, and as the formulas say."""
    import torch
    for kind in ("convex", "normalised"):
        p = problem(dev, 12, 2, 4, 96, "f32", kind)
        p["r"][:, :, ::3] = 100.0
        p["r"][:, :, 1::3] = -100.0
        p["i"][:, :, ::5] = -100.0
        p["z"][:, :, ::7] = -100.0
        p["decay"] = torch.tensor([0.0, 1.0, 0.5, 0.999] if kind == "convex" else [-120.0, -60.0, 30.0, -9.0], device=dev)
        y, h = run_fwd(ss, p)
        g = forward(p, adds(96))
        # what falls below 2^-126 is 0 in fp32, and the input's weight is a square root of such a product: at most
        # sqrt(2 * 240 * 2^-126) = 2.4e-18 off (240 = 8 softplus(30)), times values and adjoints below 400
        check("y", f64(y), g["y"], 2.0 ** -24, floor=1e-15)
        got = ss.glr_bwd(dy=torch.ones_like(y), **p)
        torch.cuda.synchronize()
        for name, v in got.items():
            assert torch.isfinite(v).all(), (kind, name)
        want = backward(p, g, np.ones(y.shape), np.zeros((2, 4)), adds(96))
        for name in ("dx", "dr", "di", "dz", "dh0"):
            check(name, f64(got[name]), want[name], 2.0 ** -24, floor=1e-15)


def test_a_nan_stays_in_its_row(ss, dev):
    import torch
    p = problem(dev, 13, 2, 9, 1000, "bf16", "normalised")
    clean, _ = run_fwd(ss, p)
    p["x"][1, 4, 500] = float("nan")
    y, h = run_fwd(ss, p)
    assert torch.isnan(y[1, 4, 500:]).all() and torch.isnan(h[1, 4])
    y[1, 4] = clean[1, 4]
    assert torch.equal(y, clean)


@pytest.mark.parametrize("kind", ["convex", "normalised"])
@pytest.mark.parametrize("L", [5, 300, 700, 2100, 9000])
def test_infinite_and_nan_biases_end_with_the_row(ss, dev, kind, L):
    """A channel whose gate's bias is infinite is open or closed at its tokens, however the row's end falls into a vector:
    the final state is the last output.  A NaN spoils its channel alone."""
    import torch
    p = problem(dev, 24, 2, 4, L, "f32", kind, z=False)
    clean, _ = run_fwd(ss, p)
    p["r_bias"] = torch.tensor([float("inf"), float("-inf"), float("nan"), float(p["r_bias"][3])], device=dev)
    y, h = run_fwd(ss, p)
    assert torch.isfinite(y[:, :2]).all() and torch.isnan(y[:, 2]).all() and torch.isnan(h[:, 2]).all()
    assert torch.equal(y[:, 3], clean[:, 3])
    kept = 0 if kind == "convex" else 1          # the gate that keeps the state
    assert torch.equal(h[:, kept], p["h0"][:, kept]) and torch.equal(y[:, kept, -1], p["h0"][:, kept])
    other = 1 - kept                              # a and u are constants of the channel: one step from the last output but one
    assert float((h[:, other] - y[:, other, -1]).abs().max()) <= 1e-5 * float(y[:, other].abs().max())


@pytest.mark.parametrize("rows,L", [(5, 33), (5, 700), (5, 1500), (5, 5003), (5, 70001), (300, 17001)])
def test_a_nan_goes_one_way(ss, dev, rows, L):
    """A NaN input spoils the outputs from its token on, a NaN upstream gradient dx up to its token, and neither any other bit,
    in the kernels for groups of lanes, for one to eight waves and for split rows."""
    import torch
    p = problem(dev, 27, 1, rows, L, "bf16", "convex", z=False)
    y0, _ = run_fwd(ss, p)
    g0 = ss.glr_bwd(dy=p["i"], **p)
    for t in (0, 7, L // 2, L - 1):
        bad = dict(p, x=p["x"].clone())
        bad["x"][0, 3, t] = float("nan")
        y, h = run_fwd(ss, bad)
        assert torch.isnan(y[0, 3, t:]).all() and torch.isnan(h[0, 3])
        y[0, 3, t:] = y0[0, 3, t:]
        assert torch.equal(y, y0)
        dy = p["i"].clone()
        dy[0, 3, t] = float("nan")
        g = ss.glr_bwd(dy=dy, **p)
        torch.cuda.synchronize()
        assert torch.isnan(g["dx"][0, 3, :t + 1]).all() and torch.isnan(g["dh0"][0, 3])
        g["dx"][0, 3, :t + 1] = g0["dx"][0, 3, :t + 1]
        assert torch.equal(g["dx"], g0["dx"])


def test_empty_sequence(ss, dev):
    import torch
    p = problem(dev, 14, 2, 3, 0, "bf16", "convex")
    y, h = run_fwd(ss, p)
    assert y.shape == (2, 3, 0) and torch.equal(h, p["h0"])
    dh = torch.randn(2, 3, device=dev)
    g = ss.glr_bwd(dy=p["x"], dh_final=dh, **p)
    torch.cuda.synchronize()
    assert torch.equal(g["dh0"], dh)
    assert not any(g[k].any() for k in ("ddecay", "dr_bias", "di_bias"))
    p["h0"] = None
    assert not run_fwd(ss, p)[1].any()


@pytest.mark.parametrize("L", [37, 2100])
def test_offsets_past_32_bits(ss, dev, L):
    """More than 2^31 elements: the last rows of a large call are bit for bit those of a call of their own."""
    import torch
    rows = (1 << 31) // L + 1000
    p = problem(dev, 25, 1, 5, L, "bf16", "convex", z=False)
    big = {k: None if v is None else torch.zeros((1, rows, L), dtype=v.dtype, device=dev) for k, v in p.items() if k in ("x", "r", "i", "z")}
    vec = {k: torch.zeros(rows, device=dev) for k in ("decay", "r_bias", "i_bias")}
    h0 = torch.zeros(1, rows, device=dev)
    for k, v in big.items():
        if v is not None:
            v[:, -5:] = p[k]
    for k, v in vec.items():
        v[-5:] = p[k]
    h0[:, -5:] = p["h0"]
    y, h = ss.glr_fwd(**big, **vec, h0=h0, kind="convex")
    y5, h5 = run_fwd(ss, p)
    assert torch.equal(y[:, -5:], y5) and torch.equal(h[:, -5:], h5) and not y[:, :-5].any()
    del y
    dy = torch.zeros_like(big["x"])
    dy[:, -5:] = p["x"]
    g = ss.glr_bwd(dy=dy, **big, **vec, h0=h0, kind="convex")
    g5 = ss.glr_bwd(dy=p["x"], **p)
    torch.cuda.synchronize()
    for k in ("dx", "dr", "di"):
        assert torch.equal(g[k][:, -5:], g5[k]), k
    for k in ("ddecay", "dr_bias", "di_bias"):
        assert torch.equal(g[k][-5:], g5[k]), k
    assert torch.equal(g["dh0"][:, -5:], g5["dh0"])


def test_channels_past_a_grid_of_sums(ss, dev):
    """Per-channel gradients of more channels than 2^22 workgroups of 32: the last ones are those of a call of their own,
    the others, whose inputs are zeros, are zeros."""
    import torch
    dim = (1 << 27) + 40
    p = problem(dev, 26, 1, 5, 1, "bf16", "convex", z=False, h0=False)
    p["i"] = p["i_bias"] = None
    wide = {k: torch.zeros((1, dim, 1), dtype=p[k].dtype, device=dev) for k in ("x", "r")}
    vec = {k: torch.zeros(dim, device=dev) for k in ("decay", "r_bias")}
    dy = torch.zeros_like(wide["x"])
    for k in wide:
        wide[k][:, -5:] = p[k]
    for k in vec:
        vec[k][-5:] = p[k]
    dy[:, -5:] = p["r"]
    g = ss.glr_bwd(dy=dy, **wide, **vec, kind="convex")
    g5 = ss.glr_bwd(dy=p["r"], **p)
    torch.cuda.synchronize()
    for k in ("ddecay", "dr_bias"):
        assert torch.equal(g[k][-5:], g5[k]) and not g[k][:-5].any(), k


def test_outputs_stay_inside_their_rows(ss, dev):
    """Nothing is written behind the last row or before the first, at lengths that end inside a vector."""
    import torch
    for L in (1, 5, 333, 2051):
        p = problem(dev, 15, 3, 5, L, "bf16", "normalised")
        n = p["x"].numel()
        flat = torch.full((n + 64,), 7.0, dtype=torch.bfloat16, device=dev)
        y = flat[32:32 + n].view(3, 5, L)
        ss.glr_fwd(**p, y=y)
        torch.cuda.synchronize()
        assert (flat[:32] == 7).all() and (flat[32 + n:] == 7).all()
        assert torch.equal(y, ss.glr_fwd(**p)[0])


def test_repeats_and_graph_replays_are_bitwise_equal(ss, dev):
    import torch
    for batch, dim, L in ((2, 64, 300), (1, 8, 9000), (1, 600, 2500)):
        p = problem(dev, 16, batch, dim, L, "bf16", "normalised")
        dy = torch.randn_like(p["x"])
        ckpt = torch.empty(ss.glr_ckpt_numel(batch, dim, L), device=dev)

        def both():
            y, h = ss.glr_fwd(**p, ckpt=ckpt)
            return dict(ss.glr_bwd(dy=dy, ckpt=ckpt, **p), y=y, h=h)

        want = {k: v.clone() for k, v in both().items()}
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            both()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        graph, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = both()
        with torch.cuda.graph(second):
            more = both()
        for k in range(3):
            for v in list(got.values()) + list(more.values()):
                v.zero_()
            graph.replay()
            second.replay()
            torch.cuda.synchronize()
            for name in want:
                assert torch.equal(got[name], want[name]) and torch.equal(more[name], want[name]), (name, k)
            again = both()
            torch.cuda.synchronize()
            assert all(torch.equal(again[n], want[n]) for n in want)


@pytest.mark.parametrize("rows,L", [(3, 2048 * 70 + 1), (2, 2048 * 130 + 5), (300, 33000)])
def test_split_rows_in_a_graph(ss, dev, rows, L):
    """Tiles of two and four pieces, and more rows than compute units: replays between eager calls, each as the first."""
    import torch
    p = problem(dev, 30, 1, rows, L, "bf16", "convex")
    dy = torch.randn_like(p["x"])

    def both():
        y, h = ss.glr_fwd(**p)
        return dict(ss.glr_bwd(dy=dy, **p), y=y, h=h)

    want = {k: v.clone() for k, v in both().items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for k in range(3):
        for v in got.values():
            v.zero_()
        graph.replay()
        eager = both()
        torch.cuda.synchronize()
        for name in want:
            assert torch.equal(got[name], want[name]) and torch.equal(eager[name], want[name]), (name, k)


def test_two_streams_at_once(ss, dev):
    import torch
    a, b = problem(dev, 17, 1, 40, 5000, "bf16", "convex"), problem(dev, 18, 1, 40, 5000, "bf16", "convex")
    ya, yb = run_fwd(ss, a)[0], run_fwd(ss, b)[0]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(s1):
            y1 = ss.glr_fwd(**a)[0]
        with torch.cuda.stream(s2):
            y2 = ss.glr_fwd(**b)[0]
        torch.cuda.synchronize()
        assert torch.equal(y1, ya) and torch.equal(y2, yb)


def test_theorem_1_gated_recurrence_equals_the_scan(ss, dev):
    """The scan with one state, A = -1, B = C = 1 and the zero-order hold is h = (1 - s(g)) h + s(g) x (Theorem 1 in the
    reader's notes): the convex recurrence with r = -g."""
    import torch
    batch, D, L = 2, 24, 700
    gen = torch.Generator().manual_seed(3)
    x, g = (torch.randn(batch, D, L, generator=gen).to(dev) for _ in range(2))
    one = torch.ones(batch, 1, L, device=dev)
    y1, h1 = ss.scan_fwd(x, g, one, one, -torch.ones(D, 1, device=dev), zoh=True)
    y2, h2 = ss.glr_fwd(x, -g, kind="convex")
    torch.cuda.synchronize()
    e = float((y1 - y2).double().norm() / y2.double().norm())
    log("scan against recurrence: rel-L2 %.2e" % e)
    assert e < 1e-5 and float((h1[..., 0] - h2).abs().max()) < 1e-4


def test_tensor_checks(ss, dev):
    import torch
    p = problem(dev, 19, 2, 3, 16, "bf16", "normalised")
    ok = dict(p)
    for change, err in ((dict(r=p["r"].float()), TypeError), (dict(r=p["r"][..., :8]), ValueError),
                        (dict(kind="other"), ValueError), (dict(decay=p["decay"].double()), TypeError),
                        (dict(h0=p["h0"].t()), ValueError), (dict(i=p["i"].transpose(1, 2).contiguous().transpose(1, 2)), ValueError),
                        (dict(decay=None), ss.SsError), (dict(i=None), ss.SsError),
                        (dict(x=p["x"].half()), TypeError), (dict(decay_scale=0.0), ss.SsError), (dict(y=p["x"]), ss.SsError)):
        with pytest.raises(err):
            ss.glr_fwd(**{**ok, **change})
    with pytest.raises(ValueError):
        ss.glr_fwd(**{k: v.cpu() if hasattr(v, "cpu") else v for k, v in p.items()})
    with pytest.raises(ValueError):
        ss.glr_bwd(dy=p["x"], workspace=torch.empty(8, dtype=torch.uint8, device=dev), **p)


# where a NaN in one operand of token t (or of the channel) goes: the tokens of each result from, up to and at t, or all of them; a
# result that is not named stays as it was
NAN_GOES = {
    "x": dict(y="from", h="all", dr="from", di="at", dz="from", ddecay="all", dr_bias="all", di_bias="all"),
    "r": dict(y="from", h="all", dx="upto", dr="all", di="upto", dz="from", ddecay="all", dr_bias="all", di_bias="all", dh0="all"),
    "i": dict(y="from", h="all", dx="at", dr="from", di="at", dz="from", ddecay="all", dr_bias="all", di_bias="all"),
    "z": dict(y="at", dx="upto", dr="upto", di="upto", dz="at", ddecay="all", dr_bias="all", di_bias="all", dh0="all"),
    "h0": dict(y="all", h="all", dr="all", dz="all", ddecay="all", dr_bias="all"),
    "i_bias": dict(y="all", h="all", dx="all", dr="all", di="all", dz="all", ddecay="all", dr_bias="all", di_bias="all"),
    "r_bias": {k: "all" for k in ("y", "h", "dx", "dr", "di", "dz", "ddecay", "dr_bias", "di_bias", "dh0")},
    "decay": {k: "all" for k in ("y", "h", "dx", "dr", "di", "dz", "ddecay", "dr_bias", "di_bias", "dh0")},
}


@pytest.mark.parametrize("rows,L,kind,io", [(5, 33, "convex", "bf16"), (5, 37, "normalised", "f32"), (5, 700, "normalised", "bf16"), (5, 1500, "convex", "f32"),
                                            (5, 5003, "normalised", "f32"), (5, 5003, "convex", "bf16"), (300, 17001, "normalised", "bf16"), (5, 2048 * 5 + 9, "convex", "f32"),
                                            (4, 2048 * 70 + 1, "normalised", "bf16"), (4, 2048 * 131 + 5, "convex", "bf16"), (321, (1 << 17) + 3, "normalised", "bf16")])
def test_where_a_nan_goes(ss, dev, rows, L, kind, io):
    """A NaN in any operand reaches exactly the results that the formulas carry it to, in every plan: groups of lanes, one to
    sixteen waves to a row, split rows in tiles of one, two and four pieces."""
    import torch
    p = problem(dev, 31, 1, rows, L, io, kind)
    dy = p["i"]

    def both(p):
        ckpt = torch.empty(ss.glr_ckpt_numel(1, rows, L), device=dev)
        y, h = ss.glr_fwd(**p, ckpt=ckpt)
        out = dict(ss.glr_bwd(dy=dy, **p), y=y, h=h)
        stored = ss.glr_bwd(dy=dy, ckpt=ckpt, **p)
        return out, dict(stored, y=y, h=h)

    clean = both(p)[0]
    for name, goes in NAN_GOES.items():
        for t in (0, L // 2 + 1, L - 1) if p[name].dim() == 3 and rows * L < 1 << 20 else (L - 2,):
            bad = dict(p, **{name: p[name].clone()})
            if bad[name].dim() == 3:
                bad[name][0, 3, t] = float("nan")
            else:
                bad[name].view(-1)[3] = float("nan")
            for got in both(bad):
                torch.cuda.synchronize()
                for k, v in got.items():
                    part = {"all": slice(None), "from": slice(t, None), "upto": slice(0, t + 1), "at": slice(t, t + 1), None: slice(0, 0)}[goes.get(k)]
                    at = (0, 3, part) if v.dim() == 3 else ((0, 3) if v.dim() == 2 else (3,))
                    if goes.get(k):
                        assert torch.isnan(v[at]).all(), (name, t, k)
                        v = v.clone()
                        v[at] = clean[k][at]
                    assert torch.equal(v, clean[k]), (name, t, k)


@pytest.mark.parametrize("L", [1, 5, 300, 700, 2100, 9000, 16391, 2048 * 70 + 1])
def test_infinite_rates_end_with_the_row(ss, dev, L):
    """A normalised channel whose rate is infinite (a decay of +inf, or one whose product with the scale overflows) forgets at every
    token and keeps the state at padding; one whose rate is zero (-inf) keeps it throughout.  Against the formulas in 64 bits,
    however the row's end falls into a vector, and the single token like the sequence."""
    import torch
    p = problem(dev, 32, 2, 4, L, "f32", "normalised", z=False)
    p["decay"] = torch.tensor([float("inf"), 1e38, float("-inf"), -3.0], device=dev)
    p["r"][:, :, 2::3] = float("-inf")           # padding
    if L > 4:
        p["r"][1, :, L - 2:] = float("-inf")
    state = p["h0"].clone()
    y, h = run_fwd(ss, p)
    dy = torch.randn(y.shape, generator=torch.Generator().manual_seed(6)).to(dev)
    dh = torch.ones(2, 4, device=dev)
    ckpt = torch.empty(ss.glr_ckpt_numel(2, 4, L), device=dev)
    ss.glr_fwd(**p, ckpt=ckpt)
    grads = [ss.glr_bwd(dy=dy, dh_final=dh, ckpt=c, **p) for c in (None, ckpt)]
    torch.cuda.synchronize()
    open_ = np.isfinite(f64(p["r"][:, :3]))
    a = np.where(np.arange(3)[:, None] < 2, 1.0 - open_, 1.0)          # exactly 0 or 1, and m is the other
    gm = lambda v: v * V(1.0 - a)  # noqa: E731
    iota = sigmoid(V(f64(p["i"][:, :3])) + V(f64(p["i_bias"][:3, None])))
    ix = V(f64(p["x"][:, :3])) * iota
    hh, _ = recur(V(a), gm(ix), V(f64(p["h0"][:, :3])), adds(L))
    check("y", f64(y[:, :3]), hh, 2.0 ** -24)
    assert torch.equal(h[:, :3], y[:, :3, -1]) and torch.isfinite(h).all() and torch.isfinite(y).all()
    G, after = recur(V(a[..., ::-1]), (V(a) * V(f64(dy[:, :3])))[..., ::-1], V(np.ones((2, 3))), adds(L))
    g = V(f64(dy[:, :3])) + after[..., ::-1]
    for got in grads:
        check("dx", f64(got["dx"][:, :3]), gm(g) * iota, 2.0 ** -24)
        check("di", f64(got["di"][:, :3]), gm(g) * ix * (V(1.0) - iota), 2.0 ** -24)
        check("dh0", f64(got["dh0"][:, :3]), G[..., -1], 2.0 ** -24)
        for k in ("dr", "ddecay", "dr_bias"):    # the decay is flat there
            v = got[k][:, :3] if got[k].dim() == 3 else got[k][:3]
            assert not v.any(), k
        assert all(torch.isfinite(v).all() for v in got.values() if v is not None)
    if L <= 5:
        for t in range(L):
            yt = ss.glr_step(state, *(p[k][..., t].contiguous() for k in ("x", "r", "i")), decay=p["decay"], r_bias=p["r_bias"],
                             i_bias=p["i_bias"])
            check("step", f64(yt[:, :3]), hh[..., t], 2.0 ** -24)
        torch.cuda.synchronize()
        assert torch.isfinite(state).all()


# Sums over tokens and batch rows of which every term counts: the gates are 0 (r = -inf) at even tokens and 1/2 (r = 0) at odd ones,
# the floor 0, the input gate 1/2, and x and dy small odd and even whole numbers, so that each term of the three sums is a multiple
# of 1/16 that is not zero (dr is, where the gate is 0), and each partial sum is exact in fp32: below 2^24 / 16 in size.  A single
# term lost, doubled or taken from another channel changes the result.
def counted(dev, batch, dim, L, io):
    import torch
    gen = torch.Generator().manual_seed(batch + L)
    dt = torch.float32 if io == "f32" else torch.bfloat16
    even = torch.arange(L) % 2 == 0

    def whole(odd):    # odd numbers from -3 to 3, or even ones from -4 to 4
        return torch.where(odd, 2 * torch.randint(-2, 2, (batch, dim, L), generator=gen) + 1, 4 * torch.randint(-1, 1, (batch, dim, L), generator=gen) + 2)

    x, dy = whole(even), whole(torch.ones(L, dtype=torch.bool))
    r = torch.where(even, -torch.inf, 0.0).expand(batch, dim, L)
    as_io = lambda t: t.to(dt).to(dev).contiguous()  # noqa: E731
    p = dict(x=as_io(x), r=as_io(r), i=torch.zeros(batch, dim, L, dtype=dt, device=dev), kind="convex", decay=torch.zeros(dim, device=dev))
    # in 64 bits: a is 0 or 1/2 and m = 1 - a
    x, dy, a = x.double().numpy(), dy.double().numpy(), torch.where(even, 0.0, 0.5).double().numpy()
    ix, before = x / 2, np.zeros_like(x)
    h = np.zeros((batch, dim))
    g, G = np.empty_like(x), np.zeros((batch, dim))
    for t in range(L):
        before[..., t] = h
        h = a[t] * h + (1 - a[t]) * ix[..., t]
    for t in range(L - 1, -1, -1):
        g[..., t] = dy[..., t] + G
        G = a[t] * g[..., t]
    dd = g * (before - ix) * (1 - a)
    terms = dict(ddecay=dd, dr_bias=dd * a, di_bias=g * (1 - a) * x / 4)
    return p, as_io(torch.from_numpy(dy)), terms


# batch rows past one pass of the sums' 32 threads, and past two; split rows of more parts than one pass of 256 threads takes
@pytest.mark.parametrize("batch,dim,L,io", [(33, 5, 37, "f32"), (70, 37, 4, "bf16"), (299, 3, 1, "f32"), (65, 2, 700, "bf16"), (2, 3, 6145, "f32"), (40, 3, 2048 * 7 + 5, "bf16"),
                                            (37, 1, 2048 * 7 + 1, "f32"), (1, 4, 2048 * 260 + 3, "bf16")])
def test_every_token_counts_in_the_sums(ss, dev, batch, dim, L, io):
    import torch
    p, dy, terms = counted(dev, batch, dim, L, io)
    ckpt = torch.empty(ss.glr_ckpt_numel(batch, dim, L), device=dev)
    ss.glr_fwd(**p, ckpt=ckpt)
    for stored in (None, ckpt):
        got = ss.glr_bwd(dy=dy, ckpt=stored, **p)
        torch.cuda.synchronize()
        for k, v in terms.items():
            there = slice(1, None, 2) if k == "dr_bias" else slice(1, None)    # token 0 has no state before it, but an input
            assert (v[..., there] != 0).all() and np.abs(v).sum((0, 2)).max() < 2 ** 20 and (v * 16 % 1 == 0).all(), k
            assert np.array_equal(f64(got[k]), v.sum((0, 2))), k


@pytest.mark.parametrize("kind,i,z", [("normalised", True, True), ("convex", False, False)])
def test_sixteen_waves_against_the_formulas(ss, dev, kind, i, z):
    """bf16 rows of 2^17 tokens and more, 321 of them so that each has a workgroup: sixteen waves forward, eight backward.  Three
    of the rows, element by element."""
    import torch
    rows, L = 321, (1 << 17) + 3
    p = problem(dev, 33, 1, rows, L, "bf16", kind, i, z)
    ckpt = torch.full((ss.glr_ckpt_numel(1, rows, L),), float("nan"), device=dev)
    y, h = ss.glr_fwd(**p, ckpt=ckpt)
    gen = torch.Generator().manual_seed(34)
    dy = torch.randn(p["x"].shape, generator=gen).to(torch.bfloat16).to(dev)
    dh = torch.randn((1, rows), generator=gen).to(dev)
    grads = [ss.glr_bwd(dy=dy, dh_final=dh, ckpt=c, **p) for c in (None, ckpt)]
    torch.cuda.synchronize()
    at = torch.tensor([0, 160, 320], device=dev)
    some = lambda t: None if t is None else t[at] if t.dim() == 1 else t[:, at]  # noqa: E731
    few = {k: some(v) if k != "kind" else v for k, v in p.items()}
    g = forward(few, adds(L))
    check("y", f64(some(y)), g["y"], HALF["bf16"])
    check("h_final", f64(some(h)), g["h"][..., -1], 0.0)
    check("ckpt", f64(some(ckpt.view(1, rows, -1))[..., 1:]), g["h"][..., 2047:L - 1:2048], 0.0)
    want = backward(few, g, f64(some(dy)), f64(some(dh)), adds(L))
    for got in grads:
        for name, v in want.items():
            check(name, f64(some(got[name])), v, HALF["bf16"] if got[name].dtype == torch.bfloat16 else 0.0)


def test_c_names_of_the_binding(ss, dev):
    """The C entry points under their own names: as the tensor calls, in place and through a workspace."""
    import torch
    B, D, L = 1, 3, 9000
    p = problem(dev, 35, B, D, L, "bf16", "normalised")
    y, h = run_fwd(ss, p)
    dy = p["i"]
    want = ss.glr_bwd(dy=dy, **p)
    s = torch.cuda.current_stream().cuda_stream
    a = lambda *names: [p[n].data_ptr() for n in names]  # noqa: E731
    new = {k: torch.empty_like(v) for k, v in dict(want, y=y, h=h).items()}
    ckpt = torch.empty(ss.ss_glr_ckpt_bytes(B, D, L) // 4, device=dev)
    ws = torch.empty(max(ss.ss_glr_fwd_workspace_bytes(B, D, L), ss.ss_glr_bwd_workspace_bytes(B, D, L)), dtype=torch.uint8, device=dev)
    head = (B, D, L, ss.SS_BF16, ss.SS_GLR_NORMALISED, SCALE)
    ins = a("x", "r", "i", "z", "decay", "r_bias", "i_bias")
    ss.ss_glr_fwd(*head, *ins, *a("h0"), new["y"].data_ptr(), new["h"].data_ptr(), ckpt.data_ptr(), ws.data_ptr(), ws.numel(), s)
    ss.ss_glr_bwd(*head, *ins, *a("h0"), dy.data_ptr(), None, ckpt.data_ptr(),
                  *(new[k].data_ptr() for k in ("dx", "dr", "di", "dz", "ddecay", "dr_bias", "di_bias", "dh0")), ws.data_ptr(), ws.numel(), s)
    torch.cuda.synchronize()
    for k, v in dict(want, y=y, h=h).items():
        assert torch.equal(new[k], v), k
    one = problem(dev, 36, 3, 5, 1, "bf16", "normalised", step=True)
    state, other = one.pop("h0"), torch.empty(3, 5, device=dev)
    out = torch.empty_like(one["x"])
    ss.ss_glr_step(3, 5, ss.SS_BF16, ss.SS_GLR_NORMALISED, SCALE, state.data_ptr(), other.data_ptr(),
                   *(one[k].data_ptr() for k in ("x", "r", "i", "z", "decay", "r_bias", "i_bias")), out.data_ptr(), s)
    again = ss.glr_step(state, **one)
    torch.cuda.synchronize()
    assert torch.equal(out, again) and torch.equal(other, state)
    with pytest.raises(ss.SsError):
        ss.ss_glr_step(3, 5, ss.SS_BF16, 7, SCALE, state.data_ptr(), other.data_ptr(), *[None] * 7, out.data_ptr(), s)
