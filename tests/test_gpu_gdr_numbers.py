"""The gated delta rule's numbers where a norm over all results does not show them: how outputs are rounded, gates and sizes at the
ends of the kernels' ranges, the gates' gradients token by token."""
import math

import pytest
import torch

from blocks import F32_REL, close, gdr64, leaves, rel, up
from test_gpu_gdr import check_bwd, check_fwd, problem, ss, want  # noqa: F401

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32
NAMES = ("q", "k", "v", "g", "beta", "h0")


@pytest.mark.parametrize("size", [(1, 1000, 2, 4, 64, 128), (2, 200, 1, 4, 128, 128), (8, 2048, 2, 16, 64, 64), (1, 90, 1, 3, 30, 50), (4, 16, 2, 2, 64, 64), (3, 600, 1, 2, 128, 200)], ids=str)
def test_bf16_outputs_are_rounded_once(ss, size):  # noqa: F811
    """bf16 outputs are fp32 results rounded once, whatever the length.  An fp32 result off by d, before a rounding to steps of s,
    leaves the 64-bit result's own rounding in a share d / s of the values, each by s: a square of d s in the mean.  With d up to
    2 F32_REL of a value (its own and the mean one's size) and s up to 2^-7 that is 2^-15 2^-7, 2^-11 of the norm."""
    p = problem(*size, BF, seed=2)
    o, _ = ss.gdr_fwd(*[p[n] for n in NAMES])
    wo, _ = want(p)
    assert rel(o, wo.to(BF).double()) <= 2.0 ** -11


@pytest.mark.parametrize("io", [F, BF])
@pytest.mark.parametrize("L", [20, 150, 450])
@pytest.mark.parametrize("qv,kv,first", [(1.5, 0.046875, (-1.99, 0.01, -0.02)), (0.09375, 0.09375, (-1.99, 0.001, -0.0111))], ids=str)
def test_parallel_rows_of_equal_values(ss, io, L, qv, kv, first):  # noqa: F811
    """Queries and keys as long as their largest value allows, all alike, under gates that decay, grow and decay by parts of a
    factor of 2 in every chunk: what a chunk's tokens read of each other is as large as its operands ever are."""
    p = problem(1, L, 1, 2, 128, 64, io)
    p["q"], p["k"] = torch.full_like(p["q"], qv), torch.full_like(p["k"], kv)
    p["g"] = torch.full((1, L, 2), -0.1)
    for n, x in enumerate(first):
        p["g"][:, n::64] = x * math.log(2.0)
    p["g"] = p["g"].cuda()
    check_fwd(ss, p)
    check_bwd(ss, p)


@pytest.mark.parametrize("io", [F, BF])
def test_gates_around_nothing(ss, io):  # noqa: F811
    """Gates of either sign in many heads, for rows of equal values: some of them turn at every place of a chunk.

    What such gates let grow is mostly at right angles to the one key there is, and not read: a head's state reaches 10^5 times what is
    read of it, and the recurrence token by token in fp32 is off by 9e-5 of o here.  F32_REL is of the sizes of a product's terms
    (see blocks.py), so here it is taken of them, token by token: |q| |S| of o, |S| |do| of dq, |k| |dS| of dv over beta, |dS| |u| and
    |S'| |dv| of dk, |dS| |S'| of dg, |dS| |k| (|v| + |S'| |k|) of dbeta; bf16's rounding (half a step, 2^-8) is of the result."""
    p = problem(1, 200, 1, 40, 128, 32, io)
    p["q"], p["k"] = torch.full_like(p["q"], 0.109375), torch.full_like(p["k"], 0.0859375)
    p["g"] = 0.3 * torch.randn(1, 200, 40, generator=torch.Generator().manual_seed(8)).cuda()
    p["beta"] *= 0.5
    gen = torch.Generator().manual_seed(1)
    do, dh = torch.randn(p["v"].shape, generator=gen).to(io).cuda(), torch.randn(p["h0"].shape, generator=gen).cuda()
    o, h = ss.gdr_fwd(*[p[n] for n in NAMES])
    got = ss.gdr_bwd(*[p[n] for n in NAMES[:5]], do, p["h0"], dh)
    ls = leaves(*[p[n] for n in NAMES])
    q, k, v, g, beta, h0 = ls
    scale, s, outs, states, faded, us = 128 ** -0.5, h0, [], [], [], []
    for t in range(200):
        f = s * torch.exp(g[:, t])[..., None, None]
        u = beta[:, t][..., None] * (v[:, t] - (f * k[:, t][..., None]).sum(-2))
        s = f + k[:, t][..., None] * u[..., None, :]
        s.retain_grad()
        outs.append((s * q[:, t][..., None]).sum(-2) * scale)
        states.append(s)
        faded.append(f.detach())
        us.append(u.detach())
    wo = torch.stack(outs, 1)
    ((wo * up(do)).sum() + (s * up(dh)).sum()).backward()
    whole = lambda x: torch.stack([y.flatten(-2).norm(dim=-1) for y in x], 1)  # noqa: E731
    size = lambda x: x.detach().norm(dim=-1)  # noqa: E731
    S, dS, F1, U = whole([x.detach() for x in states]), whole([x.grad for x in states]), whole(faded), size(torch.stack(us, 1))
    nq, nk, nv, ndo, ndv, nb = size(q), size(k), size(v), size(up(do)), size(v.grad), beta.detach()
    half = 2.0 ** -8 if io == BF else 0.0

    def within(name, x, w, terms, step=half):
        off = (x.detach().double().cpu() - w.detach()).abs()
        allowed, off = (step * size(w) + F32_REL * terms, off.norm(dim=-1)) if w.dim() == 4 else (F32_REL * terms, off)
        assert bool((off <= allowed).all()), (name, float((off / allowed).max()))
    within("o", o, wo, size(wo) + scale * nq * S)
    within("dv", got["dv"], v.grad, ndv + nb * nk * dS)
    within("dq", got["dq"], q.grad, (scale * S * ndo).sum(-1, keepdim=True))
    within("dk", got["dk"], k.grad, (dS * U + F1 * ndv).sum(-1, keepdim=True))
    within("dg", got["dg"], g.grad, dS * F1)
    within("dbeta", got["dbeta"], beta.grad, dS * nk * (nv + F1 * nk))
    close("h_final", h, s.detach(), F32_REL)
    close("dh0", got["dh0"], h0.grad, F32_REL)


@pytest.mark.parametrize("L", [150, 450])
def test_gates_that_grow_in_bf16(ss, L):  # noqa: F811
    """Log decays above 0 where values, keys and queries are bf16."""
    p = problem(1, L, 1, 2, 32, 32, BF)
    p["beta"] *= 0.2
    p["g"] = torch.where(torch.arange(L, device="cuda")[None, :, None] // 50 % 2 == 0, 0.5, -0.5).expand(1, L, 2).contiguous()
    check_fwd(ss, p)
    check_bwd(ss, p)


def sizes64(p, do, dh):
    """Norms, for every token and head, of what a backward is formed of in 64 bits: a dict of (batch, L, heads) tensors S (the state),
    dS (its gradient), F (the decayed state before the token), u, dv; the outputs, the last state, and the inputs with their gradients."""
    ls = leaves(*[p[n] for n in NAMES])
    q, k, v, g, beta, s = on = [x.detach().cuda().requires_grad_() for x in ls]
    spread = torch.arange(v.shape[2], device="cuda") // (v.shape[2] // q.shape[2])
    outs, states, faded, us = [], [], [], []
    for t in range(q.shape[1]):
        kt = k[:, t][:, spread]
        f = s * torch.exp(g[:, t])[..., None, None]
        u = beta[:, t][..., None] * (v[:, t] - (f * kt[..., None]).sum(-2))
        s = f + kt[..., None] * u[..., None, :]
        s.retain_grad()
        outs.append((s * q[:, t][:, spread][..., None]).sum(-2) * q.shape[-1] ** -0.5)
        states.append(s)
        faded.append(f.detach().flatten(-2).norm(dim=-1))
        us.append(u.detach().norm(dim=-1))
    o = torch.stack(outs, 1)
    ((o * do.cuda()).sum() + (s * dh.cuda()).sum()).backward()
    n = dict(S=torch.stack([x.detach().flatten(-2).norm(dim=-1) for x in states], 1), dS=torch.stack([x.grad.flatten(-2).norm(dim=-1) for x in states], 1),
             F=torch.stack(faded, 1), u=torch.stack(us, 1), dv=v.grad.norm(dim=-1))
    for x, y in zip(ls, on):
        x.grad = torch.zeros_like(x) if y.grad is None else y.grad.cpu()
    return {a: b.cpu() for a, b in n.items()}, o.detach().cpu(), s.detach().cpu(), ls


def left(sizes, decays, back, width):
    """What may be off in a state of `width` values, by norm, before every token and behind the last (L + 1 norms `sizes`; `back`: of a
    gradient, against the tokens).  From every chunk on: F32_REL of the state that it starts from, which decays and grows by the gates and
    is not taken back by keys as the state is (the factor of a segment is a matrix, whose errors are of its own size); what its rows
    are held to, 2^-38 of the largest, over the square root of 64 tokens 2^-35, less the balance of a token's row, half of what the gates
    have decayed till then, 2^16 at most (see gdr_device.h; against the tokens less what it is behind the largest row, the last); and a value's smallest step at the largest scale, 2^-25 of 2^-126, times rows up to 2^13, again
    over the root of 64 tokens: 2^-135."""
    L = decays.shape[1]
    out, e = torch.zeros_like(sizes), torch.zeros_like(sizes[:, 0])
    chunks = list(range(0, L, 64))
    for c in reversed(chunks) if back else chunks:
        ts = list(range(c, min(c + 64, L)))
        start = sizes[:, ts[-1] + 1 if back else ts[0]]
        low = (decays[:, ts].cumsum(1) / math.log(2.0)).clamp_max(0.0).cummin(1)[0]
        half = torch.floor((-0.5 * low).clamp(0, 16))
        floors = 2.0 ** -35 * 2.0 ** ((half - half[:, -1:]) if back else -half) * start[:, None] + 2.0 ** -135 * width ** 0.5
        e = e + F32_REL * start
        for t in reversed(ts) if back else ts:
            e = e * torch.exp(decays[:, t])
            out[:, t if back else t + 1] = e + floors[:, t - c]
        e = e + floors[:, 0 if back else -1]
    return out


def check_linear(ss, p, dh):  # noqa: F811
    """A row without values, all of which is a product with the state before, and the gradient behind: every result against 64 bits,
    within F32_REL of the sizes of the terms and what the chunks may leave."""
    o, h = ss.gdr_fwd(*[p[n] for n in NAMES])
    got = ss.gdr_bwd(*[p[n] for n in NAMES[:5]], torch.zeros_like(p["v"]), p["h0"], dh)
    n, wo, wh, ls = sizes64(p, torch.zeros(p["v"].shape, dtype=torch.float64), up(dh))
    q, k, v, g, beta, h0 = ls
    gates, b, scale = up(p["g"]), beta.detach(), q.shape[-1] ** -0.5
    before = torch.cat((up(p["h0"]).flatten(-2).norm(dim=-1)[:, None], n["S"]), 1)
    after = torch.cat((h0.grad.flatten(-2).norm(dim=-1)[:, None], n["dS"]), 1)
    width = h0.shape[-1] * h0.shape[-2]
    E, D = left(before, gates, False, width)[:, 1:], left(after, gates, True, width)
    D0, D = D[:, 0], D[:, 1:]                              # (of the last state's gradient, which is given, nothing is off)
    nq, nk = q.detach().norm(dim=-1), k.detach().norm(dim=-1)

    def within(name, x, w, allowed, least=2.0 ** -126):
        off = (x.double().cpu() - w.detach()).abs()
        off = off.flatten(allowed.dim()).norm(dim=-1) if off.dim() > allowed.dim() else off
        allowed = allowed + least                          # (results below the normal numbers)
        assert bool((off <= allowed).all()), (name, float((off / allowed).max()))
    r = F32_REL
    within("o", o, wo, scale * nq * (r * n["S"] + E))
    within("h_final", h, wh, r * n["S"][:, -1] + E[:, -1])
    within("dv", got["dv"], v.grad, r * n["dv"] + b * nk * (r * n["dS"] + D))
    # (in the last step a factor is a float, so a multiple of 2^-149, and a product's sum up to 2^35: 2^-114)
    within("dbeta", got["dbeta"], beta.grad, nk * nk * (r * n["dS"] * n["F"] + D * n["F"] + n["dS"] * E), 2.0 ** -114)
    within("dk", got["dk"], k.grad, r * (n["dS"] * n["u"] + n["F"] * n["dv"]) + D * n["u"] + E * n["dv"] + b * nk * (n["dS"] * E + n["F"] * D), 2.0 ** -114)
    within("dh0", got["dh0"], h0.grad, r * after[:, 0] + D0)


def linear(batch, L, heads, n, rate, at, size, beta):
    p = problem(batch, L, heads, heads, n, n, F, seed=6)
    p["v"].zero_()
    p["beta"] *= beta
    p["g"].zero_()
    p["g"][:, at] = rate
    p["h0"] *= size
    return p, torch.randn(p["h0"].shape, generator=torch.Generator().manual_seed(7)).cuda()


@pytest.mark.parametrize("rate,size,after", [(-0.76, 2.0 ** 110, 2.0 ** -60), (-1.0, 2.0 ** 120, 2.0 ** -60), (0.76, 2.0 ** -115, 2.0 ** -60), (1.0, 2.0 ** -100, 2.0 ** -110),
                                             (-0.76, 2.0 ** 20, 2.0 ** 60), (0.76, 2.0 ** -30, 2.0 ** -70)])
@pytest.mark.parametrize("beta", [0.0, 0.3])
def test_factors_of_segments(ss, rate, size, after, beta):  # noqa: F811
    """Segments of 128 tokens, the second of which decays or grows by e^(128 rate), a factor below 2^-126 or above 2^127."""
    p, dh = linear(1, 1024, 2, 64, rate, slice(128, 256), size, beta)
    check_linear(ss, p, dh * after)


@pytest.mark.parametrize("rate,size,after", [(-0.26, 2.0 ** 110, 2.0 ** -60), (0.26, 2.0 ** -100, 2.0 ** -100), (-0.26, 2.0 ** -10, 2.0 ** 100)])
def test_factors_of_long_segments(ss, rate, size, after):  # noqa: F811
    """The same in segments of 512 tokens whose chunks decay or grow by 2^24 each, so that every token's part of the factor counts."""
    p, dh = linear(2, 2048, 64, 16, rate, slice(512, 1024), size, 0.3)
    check_linear(ss, p, dh * after)


@pytest.mark.parametrize("L", [150, 1024])
@pytest.mark.parametrize("h0", [True, False])
def test_growth_of_nothing(ss, L, h0):  # noqa: F811
    """Gates that grow a state of zeros, or of next to nothing, by 2^46 in a chunk: it stays what it is."""
    p, dh = linear(1, L, 2, 64, 0.5, slice(64, 128), 2.0 ** -120 if h0 else 0.0, 0.5)
    check_linear(ss, p, dh * 0.0)
    p["h0"] = p["h0"] if h0 else None
    got = ss.gdr_bwd(*[p[n] for n in NAMES[:5]], torch.zeros_like(p["v"]), p["h0"], dh * 0.0)
    assert all(float(x.abs().max()) == 0.0 for x in got.values() if x is not None)
    if not h0:
        assert all(float(x.abs().max()) == 0.0 for x in ss.gdr_fwd(*[p[n] for n in NAMES]))


@pytest.mark.parametrize("sk", [2.0 ** -30, 2.0 ** -62, 2.0 ** -84])
@pytest.mark.parametrize("values", [0.0, 1.0])
@pytest.mark.parametrize("io", [F, BF])
def test_keys_of_next_to_nothing(ss, sk, values, io):  # noqa: F811
    """Keys so small that outputs are the state's alone: finite, and the state's."""
    p = problem(1, 100, 1, 2, 64, 64, io, seed=3)
    p["k"], p["v"] = (p["k"].float() * sk).to(io), p["v"] * values
    check_fwd(ss, p)


@pytest.mark.parametrize("io", [F, BF])
def test_a_single_token_of_a_far_stride(ss, io):  # noqa: F811
    """One token has no neighbour: its stride, of a slice of time-major rows, does not count, in either direction."""
    p = problem(2, 1, 1, 2, 16, 24, io)
    buf = torch.zeros(2, 1 << 22, dtype=io, device="cuda")
    far = dict(p)
    for n, at in (("q", 0), ("k", 64), ("v", 128)):
        far[n] = buf.as_strided(p[n].shape, (1 << 10, 1 << 22, p[n].shape[-1], 1), at)
        far[n].copy_(p[n])
    check_fwd(ss, far)
    check_bwd(ss, far)


def parts64(p, do, dh):
    """The 64-bit gradients, with a key's where it reads the state and where it is written apart, and what they are formed of."""
    q, k, v, g, beta, h0 = leaves(*[p[n] for n in NAMES])
    kr, kw = k.detach().clone().requires_grad_(), k.detach().clone().requires_grad_()
    hk, hv, scale = q.shape[2], v.shape[2], q.shape[-1] ** -0.5
    # a row for every value head, so that no gradient is a sum of several
    q, kr, kw = [x.detach().repeat_interleave(hv // hk, 2).requires_grad_() for x in (q, kr, kw)]
    h, out, states = h0, [], []
    for t in range(q.shape[1]):
        h = h * torch.exp(g[:, t])[..., None, None]
        u = beta[:, t][..., None] * (v[:, t] - (h * kr[:, t][..., None]).sum(-2))
        h = h + kw[:, t][..., None] * u[..., None, :]
        h.retain_grad()
        states.append(h)
        out.append((h * q[:, t][..., None]).sum(-2) * scale)
    ((torch.stack(out, 1) * do).sum() + (h * dh).sum()).backward()
    return q, kr, kw, v, g, beta, states


@pytest.mark.parametrize("case", ["plain", "bf16", "strong", "forgotten", "growing", "segments", "shared"])
def test_gates_gradients_token_by_token(ss, case):  # noqa: F811
    """dg and dbeta of every head and chunk by themselves.

    A vector of dq, or of dk where k reads (r) or is written (w), is within F32_REL of its own and its chunk's mean size; a sum over
    its K elements with a row takes that as independent roundings, |row| |vector| F32_REL / sqrt(K).  dg_t is the sum of
    q.dq - k.r - k.w over the chunk's tokens from t on, and of G <dS, S> over the K V elements of the chunk's end, dbeta_t is
    dR.v and k.r over beta; independent errors add their squares.  (F32_REL is
    the most that eight products in a row leave; a second plane that is lost in any of the three is two to ten times what is allowed.)"""
    L = {"segments": 700}.get(case, 200)
    hk, hv, dk, dv = (2, 4, 64, 48) if case == "shared" else (3, 3, 64, 48)
    p = problem(1, L, hk, hv, dk, dv, BF if case == "bf16" else F, seed=11)
    gen = torch.Generator().manual_seed(12)
    if case == "strong":
        p["g"] = (-8.0 * torch.rand(1, L, hv, generator=gen)).cuda()
    elif case == "forgotten":
        p["g"][:, ::37] = -float("inf")
    elif case == "growing":
        p["beta"] *= 0.2
        p["g"] = (0.3 * torch.randn(1, L, hv, generator=gen)).cuda()
    do, dh = torch.randn(p["v"].shape, generator=gen).to(p["v"].dtype).cuda(), torch.randn(p["h0"].shape, generator=gen).cuda()
    got = ss.gdr_bwd(*[p[n] for n in NAMES[:5]], do, p["h0"], dh)
    q, kr, kw, v, g, beta, states = parts64(p, up(do), up(dh))
    size = lambda x: x.norm(dim=-1)  # noqa: E731
    for c in range(0, L, 64):
        s = slice(c, min(c + 64, L))
        mean = lambda x: x + x.mean(1, keepdim=True)  # noqa: E731
        read = size(kr.grad[:, s])
        terms = (size(q[:, s]) * mean(size(q.grad[:, s]))) ** 2 + (size(kr[:, s]) * mean(read)) ** 2 + (size(kw[:, s]) * mean(size(kw.grad[:, s]))) ** 2
        from_here = terms.flip(1).cumsum(1).flip(1) / dk
        end = states[min(c + 63, L - 1)]
        ends = (size(end.detach().flatten(2)) * size(end.grad.flatten(2))) ** 2 / (dk * dv)
        allowed = F32_REL * (from_here + ends[:, None]).sum(1).sqrt()
        off = (got["dg"][:, s].double().cpu() - g.grad[:, s]).norm(dim=1)
        assert bool((off <= allowed).all()), ("dg", c, off, allowed)
        bt = beta.detach()[:, s]
        pieces = (size(v.detach()[:, s]) * mean(size(v.grad[:, s]) / bt)) ** 2 / dv + (size(kr[:, s]) * mean(read / bt)) ** 2 / dk
        allowed = F32_REL * pieces.sum(1).sqrt()
        off = (got["dbeta"][:, s].double().cpu() - beta.grad[:, s]).norm(dim=1)
        assert bool((off <= allowed).all()), ("dbeta", c, off, allowed)


@pytest.mark.parametrize("io", [F, BF])
@pytest.mark.parametrize("rate", [0.3, 1.0, 3.0])
@pytest.mark.parametrize("heads,K,V,L", [(1, 8, 16, 500), (1, 16, 128, 500), (1, 32, 16, 300), (2, 64, 128, 200), (2, 128, 64, 130)])
def test_gates_gradients_of_strong_decays(ss, io, rate, heads, K, V, L):  # noqa: F811
    """Where gates decay by several powers of 2 from token to token, dg is what is left of parts that tokens next to each other add and
    take back.  Both are formed of the same values of N and of M, so only the sums' own roundings stay: an element of dq, r or w is
    rounded by half a step, 2^-24 at most and 2^-24 / sqrt(3) in the mean, in each of some twelve additions of its own size, 2^-23
    together; these are independent over a row's elements and the chunk's tokens, and sized as in the test above."""
    p = problem(1, L, heads, heads, K, V, io, seed=13)
    gen = torch.Generator().manual_seed(14)
    p["g"] = (-rate * torch.nn.functional.softplus(torch.randn(1, L, heads, generator=gen))).cuda()
    do, dh = torch.randn(p["v"].shape, generator=gen).to(io).cuda(), torch.randn(p["h0"].shape, generator=gen).cuda()
    got = ss.gdr_bwd(*[p[n] for n in NAMES[:5]], do, p["h0"], dh)
    q, kr, kw, v, g, beta, states = parts64(p, up(do), up(dh))
    size = lambda x: x.norm(dim=-1)  # noqa: E731
    total = 0.0
    off = (got["dg"].double().cpu() - g.grad).norm()
    for c in range(0, L, 64):
        s = slice(c, min(c + 64, L))
        terms = (size(q[:, s]) * size(q.grad[:, s])) ** 2 + (size(kr[:, s]) * size(kr.grad[:, s])) ** 2 + (size(kw[:, s]) * size(kw.grad[:, s])) ** 2
        total += float(terms.detach().flip(1).cumsum(1).sum()) / K
        end = states[min(c + 63, L - 1)]
        total += float(((size(end.detach().flatten(2)) * size(end.grad.flatten(2))) ** 2).sum()) * (min(c + 64, L) - c) / (K * V)
    assert float(off) <= 2.0 ** -23 * total ** 0.5, (float(off), 2.0 ** -23 * total ** 0.5)


@pytest.mark.parametrize("L,heads", [(1024, 2), (2048, 40)])
@pytest.mark.parametrize("at", [(300,), (128, 255, 256), (5, 130, 131, 700)])
def test_states_forgotten_in_segments(ss, L, heads, at):  # noqa: F811
    """Segments whose factor is zero, also after it has grown by 2^180: neither the state before nor what it would have become gets by."""
    p = problem(1, L, heads, heads, 32, 32, F, seed=17)
    p["g"][:, list(at)] = -float("inf")
    check_fwd(ss, p)
    check_bwd(ss, p)
    q, dh = linear(1, L, heads, 32, 1.0, slice(128, 254), 2.0 ** -100, 0.3)
    q["g"][:, 254] = -float("inf")
    o, h = ss.gdr_fwd(*[q[n] for n in NAMES])
    assert float(h.abs().max()) == 0.0 == float(o[:, 254:].abs().max()) and bool(torch.isfinite(o).all())
    back = ss.gdr_bwd(*[q[n] for n in NAMES[:5]], torch.zeros_like(q["v"]), q["h0"], dh)
    assert float(back["dh0"].abs().max()) == 0.0 and all(bool(torch.isfinite(x).all()) for x in back.values())
