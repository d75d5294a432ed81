"""Cases of the operators around the selective scan: the gated linear recurrence and the norm and rotation of queries and keys.

``run`` computes a case's operator in its plain form (elementary torch operations in 32 bits, angles in 64), or with ``own``
through the package's calls.  ``exact`` computes it in 64 bits, by another order of operations.
"""
from __future__ import annotations

import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
#: Elements of the largest drawn recurrence, and values of the largest drawn norm; the largest listed ones cost more.
_MOST_GLR, _MOST_QK = 90_000_000, 150_000_000


# ------------------------------------------------------------------- cases ---

def listed():
    def glr(name, way, kind, io, batch, dim, seqlen, i, z, h0):
        return dict(name=name, op="glr", way=way, kind=kind, io=io, batch=batch, dim=dim, seqlen=seqlen, i=i, z=z, h0=h0)

    def qk(name, way, io, batch, seqlen, hq, hk, n, rot, interleaved, feature_major, extra, far):
        return dict(name=name, op="qk", way=way, io=io, batch=batch, seqlen=seqlen, hq=hq, hk=hk, n=n, rot=rot, interleaved=interleaved,
                    feature_major=feature_major, extra=extra, far=far)

    return [
        # one token for each of 256 sequences: a recurrent layer of a serving loop (the decode workload's width)
        glr("glr step 256x5120", "step", "normalised", "bf16", 256, 5120, 1, True, True, True),
        # a short prompt through a small layer: what a call costs
        glr("glr fwd 3x40x333 f32", "fwd", "convex", "f32", 3, 40, 333, True, False, True),
        # training or prefill of the 130M-shaped layer in fp32: a plain gated RNN
        glr("glr fwd 130M layer f32", "fwd", "convex", "f32", 8, 1536, 2048, False, False, False),
        # training or prefill of the 2.8B-shaped layer, all gates
        glr("glr fwd 2.8B layer", "fwd", "normalised", "bf16", 8, 5120, 2048, True, True, True),
        # one long sequence
        glr("glr fwd 1x2048x256K", "fwd", "normalised", "bf16", 1, 2048, 1 << 18, True, False, False),
        # the backward of the 2.8B-shaped layer
        glr("glr bwd 2.8B layer", "bwd", "normalised", "bf16", 8, 5120, 2048, True, True, True),
        # a training step on one long sequence of few channels (a shard of a layer), rows of odd length
        glr("glr train 1x96x300001 f32", "train", "convex", "f32", 1, 96, 300_001, True, False, True),
        # B and C of one token for each of 256 sequences, each at its own position
        qk("qk decode B, C 256", "fwd", "bf16", 256, 1, 1, 1, 16, 16, False, True, 160, True),
        # B and C of the 2.8B-shaped layer, cut from the rows of its projection (160 columns of dt before them)
        qk("qk fwd B, C 2.8B layer", "fwd", "bf16", 8, 2048, 1, 1, 16, 16, False, True, 160, False),
        # B and C of a million-token sequence of the long workload (128 columns of dt)
        qk("qk fwd B, C 1M tokens", "fwd", "bf16", 1, 1 << 20, 1, 1, 16, 8, True, True, 128, False),
        # queries and keys of an attention layer between the recurrent ones, 32 heads that share 8
        qk("qk fwd 32+8 heads of 128", "fwd", "bf16", 8, 2048, 32, 8, 128, 128, False, False, 1024, False),
        # a training step's backward of the same in fp32, heads of 80 with part of each rotated, odd length
        qk("qk bwd 20+5 heads of 80", "bwd", "f32", 4, 2047, 20, 5, 80, 32, True, False, 400, True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    if rng.random() < 0.55:
        way = rng.choice(["fwd", "fwd", "bwd", "train", "step"])
        seqlen = 1 if way == "step" else _log(rng, 1, 1 << 18)
        rows = _log(rng, 16, max(16, min(1 << 20, (_MOST_GLR if way in ("fwd", "step") else _MOST_GLR // 2) // seqlen)))
        batch = _log(rng, 1, min(rows, 300))
        return dict(op="glr", way=way, kind=rng.choice(["convex", "normalised"]), io=rng.choice(["f32", "bf16"]), batch=batch, dim=max(1, rows // batch),
                    seqlen=seqlen, i=rng.random() < 0.6, z=rng.random() < 0.4, h0=way == "step" or rng.random() < 0.5)
    way, fm = rng.choice(["fwd", "fwd", "bwd"]), rng.random() < 0.5
    if fm:
        n, hq, hk = rng.choice([2, 4, 8, 16]), rng.choice([1, 1, 2]), 1
    else:
        n, hk = rng.choice([16, 40, 64, 72, 80, 96, 128, 192, 256]), rng.choice([1, 2, 3, 5, 8])
        hq = hk * rng.choice([1, 1, 2, 4, 5])
    tokens = _log(rng, 1, min(1 << 20, _MOST_QK // ((hq + hk) * n * (1 if way == "fwd" else 2))))
    batch = _log(rng, 1, min(tokens, 300))
    return dict(op="qk", way=way, io=rng.choice(["f32", "bf16"]), batch=batch, seqlen=max(1, tokens // batch), hq=hq, hk=hk, n=n,
                rot=rng.choice([n, n, n // 2 // 2 * 2]), interleaved=rng.random() < 0.4, feature_major=fm, extra=rng.choice([0, 7, 64, 160]), far=rng.random() < 0.5)


def work(case):
    eb = 4 if case["io"] == "f32" else 2
    if case["op"] == "glr":
        n = case["batch"] * case["dim"] * case["seqlen"]
        ins = 2 + case["i"] + case["z"]          # x, r and the gates that are there
        state = case["batch"] * case["dim"] * 4
        if case["way"] == "step":
            return {"bytes": n * (ins + 1) * eb + 2 * state, "flops": 40 * n}
        if case["way"] == "fwd":
            return {"bytes": n * (ins + 1) * eb + state * (1 + case["h0"]), "flops": 40 * n}
        outs = ins + (case["way"] == "train")    # a gradient for each input, and y
        return {"bytes": n * (ins + 1 + outs) * eb + state * 4, "flops": (80 if case["way"] == "bwd" else 120) * n}
    n = case["batch"] * case["seqlen"] * (case["hq"] + case["hk"]) * case["n"]
    pos = case["batch"] * case["seqlen"] * 8 if case["far"] else 0
    if case["way"] == "fwd":
        return {"bytes": 2 * n * eb + pos, "flops": 8 * n}
    return {"bytes": 3 * n * eb + pos, "flops": 20 * n}


# ------------------------------------------------------------------ inputs ---

def prepare(case, seed):
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    io = _DT[case["io"]]

    def normal(*shape, scale=1.0, shift=0.0, dtype=torch.float32):
        v = torch.randn(shape, generator=gen, device=dev, dtype=dtype)
        return v if scale == 1.0 and shift == 0.0 else v.mul_(scale).add_(shift)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device=dev)

    s = dict(case=dict(case))
    if case["op"] == "glr":
        batch, dim, seqlen = case["batch"], case["dim"], case["seqlen"]
        full = (batch, dim) if case["way"] == "step" else (batch, dim, seqlen)
        s["x"] = normal(*full, dtype=io)
        s["r"] = normal(*full, dtype=io)
        s["i"] = normal(*full, dtype=io) if case["i"] else None
        s["z"] = normal(*full, dtype=io) if case["z"] else None
        if case["kind"] == "convex":
            s["decay"] = 0.98 * uniform(dim)                      # floors of the decay
            s["r_bias"] = normal(dim, shift=2.0)                  # gates that mostly keep the state
        else:                                                     # decays between 0.9 and 0.999 where the gate is open
            rate = -torch.log(0.9 + 0.099 * uniform(dim))
            s["decay"] = torch.log(torch.expm1(rate / 8.0))
            s["r_bias"] = normal(dim)
        s["i_bias"] = normal(dim) if case["i"] else None
        s["h0"] = normal(batch, dim) if case["h0"] else None
        if case["way"] in ("bwd", "train"):
            s["dy"] = normal(*full, dtype=io)
            s["dh_final"] = normal(batch, dim)
        return s
    batch, seqlen, hq, hk, n = (case[k] for k in ("batch", "seqlen", "hq", "hk", "n"))
    # q and k are columns of the rows that a projection wrote, behind `extra` others; C comes behind B
    rows = normal(batch, seqlen, case["extra"] + (hq + hk) * n, dtype=io)
    at = case["extra"]
    if case["feature_major"]:
        k, q = rows[..., at:at + hk * n], rows[..., at + hk * n:]
    else:
        q, k = rows[..., at:at + hq * n], rows[..., at + hq * n:]
    s["q"], s["k"] = q.unflatten(-1, (hq, n)), k.unflatten(-1, (hk, n))
    s["wq"], s["wk"] = normal(n, scale=0.2, shift=1.0), normal(n, scale=0.2, shift=1.0)
    pairs = case["rot"] // 2
    s["freq"] = 10000.0 ** (-torch.arange(pairs, device=dev, dtype=torch.float64) / max(1, pairs))
    s["pos"] = torch.randint(0, 1 << 20, (batch, seqlen), generator=gen, device=dev) if case["far"] else None
    if case["way"] == "bwd":
        def like(h):
            return normal(batch, h, n, seqlen, dtype=io) if case["feature_major"] else normal(batch, seqlen, h, n, dtype=io)
        s["dq"], s["dk"] = like(hq), like(hk)
    return s


# --------------------------------------------------------------- own calls ---

def _run_own(s):
    import selective_state_space_62_amd as ss
    c = s["case"]
    if c["op"] == "glr":
        gates = dict(i=s["i"], z=s["z"], decay=s["decay"], r_bias=s["r_bias"], i_bias=s["i_bias"], kind=c["kind"])
        if c["way"] == "step":
            state = torch.empty_like(s["h0"])
            return dict(y=ss.glr_step(s["h0"], s["x"], s["r"], state_out=state, **gates), state=state)
        if c["way"] == "fwd":
            y, h = ss.glr_fwd(s["x"], s["r"], h0=s["h0"], **gates)
            return dict(y=y, h_final=h)
        out, ckpt = {}, None
        if c["way"] == "train":
            ckpt = torch.empty(ss.glr_ckpt_numel(c["batch"], c["dim"], c["seqlen"]), dtype=torch.float32, device=s["x"].device)
            out["y"], out["h_final"] = ss.glr_fwd(s["x"], s["r"], h0=s["h0"], ckpt=ckpt, **gates)
        g = ss.glr_bwd(s["x"], s["r"], s["dy"], h0=s["h0"], dh_final=s["dh_final"], ckpt=ckpt, **gates)
        out.update({k: v for k, v in g.items() if v is not None})
        return out
    kw = dict(wq=s["wq"], wk=s["wk"], positions=s["pos"], interleaved=c["interleaved"], feature_major=c["feature_major"])
    if c["way"] == "fwd":
        q, k = ss.qk_norm_rot(s["q"], s["k"], s["freq"], **kw)
        return dict(q=q, k=k)
    return ss.qk_norm_rot_bwd(s["q"], s["k"], s["freq"], s["dq"], s["dk"], **kw)


# -------------------------------------------------------------- plain form ---

def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _softplus(v):
    return torch.clamp(v, min=0.0) + torch.log1p(torch.exp(-torch.abs(v)))


def _scan(a, u):
    """h_t = a_t h_(t-1) + u_t along the last axis from zero, by doubling: every step joins neighbours twice as far apart."""
    a, u, d = a.clone(), u.clone(), 1
    while d < a.shape[-1]:
        u[..., d:] = a[..., d:] * u[..., :-d] + u[..., d:]
        a[..., d:] = a[..., d:] * a[..., :-d]
        d *= 2
    return u


def _glr_gates(s, column):
    """The gates in 32 bits: sigmoid of r, the decay, the input's weight, the input gate (or None)."""
    c = s["case"]
    sig = _sigmoid(s["r"].float() + column(s["r_bias"]))
    if c["kind"] == "convex":
        f = column(s["decay"])
        a = f + (1.0 - f) * sig
        m = (1.0 - f) * _sigmoid(-(s["r"].float() + column(s["r_bias"])))
    else:
        rate = column(8.0 * _softplus(s["decay"]))
        a = torch.exp(-rate * sig)
        m = torch.sqrt(-torch.expm1(-2.0 * rate * sig))
    return sig, a, m, _sigmoid(s["i"].float() + column(s["i_bias"])) if c["i"] else None


def _gate_out(s, h):
    if s["z"] is None:
        return h
    z = s["z"].float()
    return h * (z * _sigmoid(z))


def _plain_glr(s):
    c, io = s["case"], s["x"].dtype
    if c["way"] == "step":
        _, a, m, iota = _glr_gates(s, lambda v: v)
        x = s["x"].float()
        state = a * s["h0"] + m * (x if iota is None else iota * x)
        return dict(y=_gate_out(s, state).to(io), state=state)
    column = lambda v: v[:, None]  # noqa: E731
    sig, a, m, iota = _glr_gates(s, column)
    x = s["x"].float()
    ix = x if iota is None else iota * x
    u = m * ix
    if s["h0"] is not None:
        u[..., 0] += a[..., 0] * s["h0"]
    h = _scan(a, u)
    del u
    out = {}
    if c["way"] in ("fwd", "train"):
        out.update(y=_gate_out(s, h).to(io), h_final=h[..., -1].clone())
        if c["way"] == "fwd":
            return out
    dy = s["dy"].float()
    w = dy.clone() if s["z"] is None else _gate_out(s, dy)   # not the input itself, to which the next line would add
    w[..., -1] += s["dh_final"]
    # g_t = w_t + a_(t+1) g_(t+1): the same scan from the other end
    g = _scan(torch.nn.functional.pad(a[..., 1:], (0, 1)).flip(-1), w.flip(-1)).flip(-1)
    del w
    before = torch.cat((torch.zeros_like(h[..., :1]) if s["h0"] is None else s["h0"][..., None], h[..., :-1]), -1)
    if c["kind"] == "convex":
        da = g * (before - ix)
        dr = da * m * sig
        ddecay = (da * (m / (1.0 - column(s["decay"])))).sum((0, 2))
    else:
        rate = column(8.0 * _softplus(s["decay"]))
        t = g * a * (a * (rate * sig / m) * ix - rate * sig * before)
        dr = (1.0 - sig) * t
        ddecay = t.sum((0, 2)) * _sigmoid(s["decay"]) / _softplus(s["decay"])
    gm = g * m
    out.update(dx=(gm if iota is None else gm * iota).to(io), dr=dr.to(io), ddecay=ddecay, dr_bias=dr.sum((0, 2)), dh0=a[..., 0] * g[..., 0])
    if iota is not None:
        di = gm * x * iota * (1.0 - iota)
        out.update(di=di.to(io), di_bias=di.sum((0, 2)))
    if s["z"] is not None:
        z = s["z"].float()
        sz = _sigmoid(z)
        out["dz"] = (dy * h * (sz * (1.0 + z * (1.0 - sz)))).to(io)
    return out


def _angles(s):
    """cos and sin of every token's angles (batch, seqlen, 1, rot/2): the products in 64 bits."""
    c = s["case"]
    pos = s["pos"] if s["pos"] is not None else torch.arange(c["seqlen"], device=s["q"].device).expand(c["batch"], -1)
    ang = pos[..., None, None].double() * s["freq"]
    return torch.cos(ang).float(), torch.sin(ang).float()


def _pairs(v, case):
    """The two halves of every rotated pair, and the rest."""
    rot = case["rot"]
    if case["interleaved"]:
        return v[..., 0:rot:2], v[..., 1:rot:2], v[..., rot:]
    return v[..., :rot // 2], v[..., rot // 2:rot], v[..., rot:]


def _joined(v1, v2, rest, case):
    head = torch.stack((v1, v2), -1).flatten(-2) if case["interleaved"] else torch.cat((v1, v2), -1)
    return torch.cat((head, rest), -1)


def _plain_qk(s):
    c = s["case"]
    cos, sin = _angles(s)
    out = {}
    for name, w in (("q", s["wq"]), ("k", s["wk"])):
        v = s[name].float()
        rho = 1.0 / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-6)
        if c["way"] == "fwd":
            n1, n2, rest = _pairs(v * rho * w, c)
            o = _joined(n1 * cos - n2 * sin, n2 * cos + n1 * sin, rest, c).to(s[name].dtype)
            out[name] = o.permute(0, 2, 3, 1).contiguous() if c["feature_major"] else o
            continue
        do = s["d" + name].float()
        d1, d2, rest = _pairs(do.permute(0, 3, 1, 2) if c["feature_major"] else do, c)
        dn = _joined(d1 * cos + d2 * sin, d2 * cos - d1 * sin, rest, c)
        out["dw" + name] = (dn * v * rho).sum((0, 1, 2))
        p = dn * w
        out["d" + name] = (rho * p - v * (rho * rho * rho * (p * v).mean(-1, keepdim=True))).to(s[name].dtype)
    return out


def run(state):
    if own:
        return _run_own(state)
    return _plain_glr(state) if state["case"]["op"] == "glr" else _plain_qk(state)


# --------------------------------------------------------------- in 64 bits ---

def _recur64(a, u):
    """h_t = a_t h_(t-1) + u_t from zero, token by token within pieces of the row and then over the pieces' ends."""
    length, piece = a.shape[-1], 64
    if length <= piece:
        h = torch.empty_like(u)
        last = torch.zeros_like(u[..., 0])
        for t in range(length):
            last = a[..., t] * last + u[..., t]
            h[..., t] = last
        return h
    full = -(-length // piece) * piece
    ap = torch.nn.functional.pad(a, (0, full - length)).unflatten(-1, (-1, piece))
    h = torch.nn.functional.pad(u, (0, full - length)).unflatten(-1, (-1, piece)).contiguous()
    reach = ap.contiguous().clone()
    for t in range(1, piece):
        h[..., t] += ap[..., t] * h[..., t - 1]
        reach[..., t] *= reach[..., t - 1]
    ends = _recur64(reach[..., -1].contiguous(), h[..., -1].contiguous())
    h[..., 1:, :] += reach[..., 1:, :] * ends[..., :-1, None]
    return h.flatten(-2)[..., :length].contiguous()


def _exact_glr(s):
    c = s["case"]
    up = lambda v: None if v is None else v.double()  # noqa: E731
    step = c["way"] == "step"
    x, r, i, z = (up(s[k]) if not step or s[k] is None else up(s[k])[..., None] for k in ("x", "r", "i", "z"))
    decay, rb, ib = (None if s[k] is None else up(s[k])[:, None] for k in ("decay", "r_bias", "i_bias"))
    sig = torch.special.expit(r + rb)
    if c["kind"] == "convex":
        keep = decay + (1 - decay) * sig
        put = (1 - decay) * torch.special.expit(-(r + rb))
    else:
        rate = 8 * torch.logaddexp(decay, torch.zeros_like(decay)) * sig
        keep, put = torch.exp(-rate), (-torch.expm1(-2 * rate)).sqrt()
    inp = x if i is None else x * torch.special.expit(i + ib)
    u = put * inp
    h0 = up(s["h0"]) if s["h0"] is not None else torch.zeros_like(u[..., 0])
    u[..., 0] += keep[..., 0] * h0
    h = _recur64(keep, u)
    del u
    sz = None if z is None else torch.special.expit(z)
    y = h if z is None else h * z * sz
    if step:
        return dict(y=y[..., 0], state=h[..., 0])
    out = {} if c["way"] == "bwd" else dict(y=y, h_final=h[..., -1])
    if c["way"] == "fwd":
        return out
    del y
    dy = up(s["dy"])
    w = dy.clone() if z is None else dy * z * sz
    w[..., -1] += up(s["dh_final"])
    back = torch.zeros_like(keep)
    back[..., 1:] = keep[..., 1:].flip(-1)
    g = _recur64(back, w.flip(-1)).flip(-1)
    prev = torch.cat((h0[..., None], h[..., :-1]), -1)
    if c["kind"] == "convex":
        dkeep = g * prev - g * inp                       # of the decay, the input's weight being 1 - decay
        dr = dkeep * (1 - decay) * sig * (1 - sig)
        ddecay = (dkeep * (1 - sig)).sum((0, 2))
    else:
        dlog = g * prev * keep - g * inp * keep * keep / put   # of the decay's logarithm
        dr = -dlog * rate * (1 - sig)
        ddecay = (-8 * dlog * sig).sum((0, 2)) * torch.special.expit(decay[:, 0])
    out.update(dr=dr, ddecay=ddecay, dr_bias=dr.sum((0, 2)), dh0=g[..., 0] * keep[..., 0])
    if i is None:
        out["dx"] = g * put
    else:
        si = torch.special.expit(i + ib)
        out["dx"] = g * put * si
        out["di"] = g * put * x * si * (1 - si)
        out["di_bias"] = out["di"].sum((0, 2))
    if z is not None:
        out["dz"] = dy * h * (sz + z * sz * (1 - sz))
    return out


def _exact_qk(s):
    """The rotation as a product of complex numbers."""
    c = s["case"]
    rot, half = c["rot"], c["rot"] // 2
    pos = s["pos"].double() if s["pos"] is not None else torch.arange(c["seqlen"], device=s["q"].device, dtype=torch.float64).expand(c["batch"], -1)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=pos.device), pos[..., None, None] * s["freq"])
    order = torch.arange(c["n"], device=pos.device)     # where the values of pair after pair stand
    if not c["interleaved"] and half:
        order = torch.cat((torch.stack((order[:half], order[half:rot]), -1).flatten(), order[rot:]))

    def turned(v, by):
        v = v[..., order]
        if half:
            t = torch.view_as_real(torch.view_as_complex(v[..., :rot].unflatten(-1, (half, 2)).contiguous()) * by).flatten(-2)
            v = torch.cat((t, v[..., rot:]), -1)
        return v[..., torch.argsort(order)]

    out = {}
    for name, w in (("q", s["wq"].double()), ("k", s["wk"].double())):
        v = s[name].double()
        size = (v.square().sum(-1, keepdim=True) / c["n"] + 1e-6).sqrt()
        unit = v / size
        if c["way"] == "fwd":
            o = turned(unit * w, turn)
            out[name] = o.permute(0, 2, 3, 1) if c["feature_major"] else o
        else:
            do = s["d" + name].double()
            dn = turned(do.permute(0, 3, 1, 2) if c["feature_major"] else do, turn.conj())
            out["dw" + name] = (dn * unit).flatten(0, 2).sum(0)
            out["d" + name] = (dn * w - unit * (dn * w * unit).sum(-1, keepdim=True) / c["n"]) / size
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_glr(s) if case["op"] == "glr" else _exact_qk(s)
