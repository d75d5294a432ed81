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
