"""Cases of the operators around the attention core: rotary positions, norms
of queries and keys with the rotation in the same pass, and causal attention
with a sliding window and sink tokens.

Where ``own`` is false, ``run`` computes them in plain torch operations in 32
bits (angles in 64); where it is true, ``run`` calls the library.
"""

import math

import torch

own = False

DEV = "cuda"
THETA = 500000.0


# ------------------------------------------------------------------- cases

def listed():
    return [
        # One new token of a long sequence: launch latency is all there is.
        dict(name="rope one token", op="rope", back=False, L=1, H=32, Hkv=8, d=128, rot=128, layout="half",
             scaling="none", pos0=262143, packed=False, fused=False),
        # A rank's rows of a sequence-sharded 131072-token input, read from the fused QKV projection's
        # output, positions scaled by frequency bands for a context beyond the trained one.
        dict(name="rope sequence shard", op="rope", back=False, L=32768, H=64, Hkv=8, d=128, rot=128, layout="half",
             scaling="bands", pos0=65536, packed=False, fused=True),
        # Gradients of packed documents (positions restart), half of each head rotated, interleaved pairs.
        dict(name="rope packed backward", op="rope", back=True, L=20011, H=32, Hkv=8, d=128, rot=64,
             layout="interleaved", scaling="linear", pos0=0, packed=True, fused=False),
        # One new token through norm and rotation.
        dict(name="norm one token", op="norm", back=False, L=1, H=64, Hkv=8, d=128, rot=128, layout="half",
             scaling="none", pos0=131071, packed=False, fused=False),
        # The 8B-shaped layer's queries and keys, forward, from the fused projection's output.
        dict(name="norm forward", op="norm", back=False, L=32768, H=32, Hkv=8, d=128, rot=128, layout="half",
             scaling="none", pos0=0, packed=False, fused=True),
        # Their gradients, with the weights' gradients.
        dict(name="norm backward", op="norm", back=True, L=32768, H=32, Hkv=8, d=128, rot=128, layout="half",
             scaling="none", pos0=0, packed=False, fused=False),
        # A short ragged batch of narrow heads, part of each rotated, interleaved: gradients.
        dict(name="norm ragged backward", op="norm", back=True, L=1025, H=6, Hkv=2, d=96, rot=48,
             layout="interleaved", scaling="none", pos0=17, packed=True, fused=False),
        # A short prompt with a window inside one tile: forward and gradients, latency bound.
        dict(name="window short", op="window", back=True, L=300, H=4, Hkv=1, W=100, S=4),
        # The 8B-shaped layer's heads, window 4096 and four sink tokens: forward alone (evaluation).
        dict(name="window forward", op="window", back=False, L=32768, H=32, Hkv=8, W=4096, S=4),
        # The same as a training step.
        dict(name="window train", op="window", back=True, L=32768, H=32, Hkv=8, W=4096, S=4),
        # One chunk (U = 8 heads of one KV head) of the 32B-shaped layer at 131072 tokens, narrow window.
        dict(name="window chunk", op="window", back=True, L=131072, H=8, Hkv=1, W=1024, S=16),
        # Ragged length and window, no sinks.
        dict(name="window ragged", op="window", back=True, L=8191, H=8, Hkv=2, W=513, S=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["rope", "norm", "window", "window"])
    if op == "window":
        while True:
            Hkv, g = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8])
            L, W = _log(rng, 1, 131072), _log(rng, 1, 8192)
            # no dearer than the dearest listed case, and its plain form's scores fit the card
            if L * W * g <= 32768 * 4096 * 8 and L * W * g * Hkv <= 32768 * 4096 * 32 and L * g * Hkv <= 1 << 20:
                return dict(op=op, back=rng.random() < 0.6, L=L, H=g * Hkv, Hkv=Hkv, W=W,
                            S=rng.choice([0, 0, 1, 4, 16, _log(rng, 1, 300)]))
    d = rng.choice([64, 72, 80, 96, 128, 128, 128, 192, 256])
    rot = rng.choice([d, d, d // 2, 2 * rng.randint(1, d // 2)])
    Hkv, g = rng.choice([1, 2, 3, 8]), rng.choice([1, 3, 4, 8])
    while True:
        L = _log(rng, 1, 65536)
        if L * (g + 1) * Hkv * d <= 32768 * 72 * 128:
            return dict(op=op, back=rng.random() < 0.5, L=L, H=g * Hkv, Hkv=Hkv, d=d, rot=rot - rot % 2,
                        layout=rng.choice(["half", "interleaved"]),
                        scaling=rng.choice(["none", "linear", "bands"]), pos0=rng.choice([0, 1, _log(rng, 1, 1 << 20)]),
                        packed=rng.random() < 0.3, fused=rng.random() < 0.5)


def work(case):
    L, H, Hkv = case["L"], case["H"], case["Hkv"]
    if case["op"] == "window":
        d, W, S = 128, min(case["W"], L), min(case["S"], L)
        seen = W * L - W * (W - 1) // 2                     # keys inside the window
        n = max(0, L - W)                                   # queries whose window has left the first token
        seen += min(n, S) * (min(n, S) + 1) // 2 + max(0, n - S) * S
        b = 2 * L * d * (2 * H + 2 * Hkv) + 4 * H * L
        if case["back"]:
            b += 2 * L * d * (2 * H + 2 * Hkv)
        return dict(bytes=b, flops=seen * H * d * (14 if case["back"] else 4))
    e = L * (H + Hkv) * case["d"]
    pos = 4 * L if case["packed"] else 0
    turn = 3 * L * (H + Hkv) * case["rot"]
    if case["op"] == "rope":
        return dict(bytes=4 * e + pos, flops=turn)
    return dict(bytes=(6 if case["back"] else 4) * e + pos + (16 if case["back"] else 8) * case["d"],
                flops=turn + (12 if case["back"] else 4) * e)


# ------------------------------------------------------------------- inputs

def _scaling(case):
    return {"none": None, "linear": ("linear", 4.0), "bands": ("bands", 8.0, 1.0, 4.0, 8192)}[case["scaling"]]


def _normal(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    L, H, Hkv = case["L"], case["H"], case["Hkv"]
    s = dict(case=case)
    if case["op"] == "window":
        s["q"], s["k"], s["v"] = _normal(g, L, H, 128), _normal(g, L, Hkv, 128), _normal(g, L, Hkv, 128)
        if case["back"]:
            s["do"] = _normal(g, L, H, 128)
        if own:
            from headwise_chunked_context_gb300 import upipe
            s["cfg"] = upipe.WindowConfig(L=L, H=H, Hkv=Hkv, window=case["W"], sinks=case["S"])
        return s
    d = case["d"]
    if case["fused"]:
        qkv = _normal(g, L, H + 2 * Hkv, d)
        s["q"], s["k"] = qkv[:, :H], qkv[:, H:H + Hkv]
    else:
        s["q"], s["k"] = _normal(g, L, H, d), _normal(g, L, Hkv, d)
    if case["packed"]:  # documents of up to 4096 tokens behind one another
        cut = torch.randint(1, 4097, (L,), generator=g, device=DEV).cumsum(0)
        at = torch.arange(L, device=DEV)
        n = torch.searchsorted(cut, at, right=True)
        start = torch.where(n > 0, cut[(n - 1).clamp(min=0)], 0)
        s["positions"] = (at - start + case["pos0"]).to(torch.int32)
    else:
        s["positions"] = None
    if case["op"] == "norm":
        s["wq"] = 1.0 + 0.1 * torch.randn(d, generator=g, device=DEV)
        s["wk"] = 1.0 + 0.1 * torch.randn(d, generator=g, device=DEV)
        if case["back"]:
            s["dq"], s["dk"] = _normal(g, L, H, d), _normal(g, L, Hkv, d)
    s["freqs"] = torch.tensor(_freqs(case["rot"], case["scaling"]), dtype=torch.float64, device=DEV)
    if own:
        from headwise_chunked_context_gb300 import upipe
        s["rope"] = upipe.Rope(d, rot=case["rot"], layout=case["layout"], theta=THETA, scaling=_scaling(case))
    return s


def _freqs(rot, scaling):
    f = [THETA ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        f = [x / 4.0 for x in f]
    if scaling == "bands":  # kept above 4 turns in 8192 tokens, divided by 8 below 1, blended between
        keep = [min(1.0, max(0.0, (8192 * x / (2 * math.pi) - 1.0) / 3.0)) for x in f]
        f = [x * (k + (1 - k) / 8.0) for x, k in zip(f, keep)]
    return f


# --------------------------------------------------------------- plain form

def _angles(s):
    c = s["case"]
    p = s["positions"] if s["positions"] is not None else torch.arange(c["L"], device=DEV) + c["pos0"]
    a = p.double()[:, None] * s["freqs"]
    return a.cos().float()[:, None], a.sin().float()[:, None]


def _turn(x, cos, sin, case):
    """Rotates the pairs of x [L, heads, d], fp32."""
    rot = case["rot"]
    y = x.clone()
    if case["layout"] == "half":
        a, b = slice(0, rot // 2), slice(rot // 2, rot)
    else:
        a, b = slice(0, rot, 2), slice(1, rot, 2)
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., a] * sin + x[..., b] * cos
    return y


def _norm_forward(x, w, cos, sin, case):
    x = x.float()
    return _turn(x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w, cos, sin, case).to(torch.bfloat16)


def _norm_backward(x, w, dy, cos, sin, case):
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
    n = x * r
    dz = _turn(dy.float(), cos, -sin, case)
    dw = (dz * n).sum((0, 1))
    dn = dz * w
    return (r * (dn - n * (dn * n).mean(-1, keepdim=True))).to(torch.bfloat16), dw


def _window_head(q, k, v, do, W, S):
    """One KV head with its g query heads, in bands: q [L, g, d], k, v [L, d]."""
    L, g, d = q.shape
    scale = 1.0 / math.sqrt(d)
    W, S = min(W, L), min(S, L)
    B = 64
    while B < 1024 and B < W:
        B *= 2
    nb = -(-L // B)
    R = -(-(W - 1) // B) * B
    pad = torch.nn.functional.pad

    def rows(x):  # [L, g, d] -> [nb, g B, d]
        x = pad(x.float(), (0, 0, 0, 0, 0, nb * B - L))
        return x.view(nb, B, g, d).transpose(1, 2).reshape(nb, g * B, d)

    def slabs(x):  # [L, d] -> [nb, d, R + B], the keys that a band may see
        return pad(x.float(), (0, 0, R, nb * B - L)).unfold(0, R + B, B)

    qb, kb, vb = rows(q), slabs(k), slabs(v)
    i = torch.arange(nb * B, device=DEV).view(nb, B, 1)
    j = (torch.arange(nb, device=DEV) * B - R).view(nb, 1, 1) + torch.arange(R + B, device=DEV)
    hidden = (j < 0) | (j > i) | (i - j >= W)
    s = (qb @ kb).mul_(scale).view(nb, g, B, R + B).masked_fill_(hidden[:, None], -math.inf).view(nb, g * B, R + B)
    m = s.amax(-1, keepdim=True)
    if S:
        ks, vs = k[:S].float(), v[:S].float()
        js = torch.arange(S, device=DEV)
        hid = (i - js < W)
        ss = (qb @ ks.T).mul_(scale).view(nb, g, B, S).masked_fill_(hid[:, None], -math.inf).view(nb, g * B, S)
        m = torch.maximum(m, ss.amax(-1, keepdim=True))
        ps = torch.exp(ss - m)
    p = torch.exp(s.sub_(m))
    del s
    z = p.sum(-1, keepdim=True)
    if S:
        z = z + ps.sum(-1, keepdim=True)
        ps = ps / z
    p = p.div_(z)
    o = p @ vb.transpose(1, 2)
    if S:
        o = o + ps @ vs

    def back(x):  # [nb, g B, c] -> [L, g, c]
        return x.view(nb, g, B, -1).transpose(1, 2).reshape(nb * B, g, -1)[:L]

    out = [back(o).to(torch.bfloat16), back(m + torch.log(z))[..., 0].t().contiguous()]
    if do is None:
        return out
    db = rows(do)
    delta = (o * db).sum(-1, keepdim=True)

    def fold(x):  # [nb, R + B, d] -> [L, d]: adds what the bands say of each key
        y = torch.zeros(nb + R // B, B, d, device=DEV)
        x = x.view(nb, R // B + 1, B, d)
        for t in range(R // B + 1):
            y[t:t + nb] += x[:, t]
        return y.view(-1, d)[R:R + L]

    dv = fold(p.transpose(1, 2) @ db)
    ds = (db @ vb).sub_(delta).mul_(p)
    del p
    dq = ds @ kb.transpose(1, 2)
    dk = fold(ds.transpose(1, 2) @ qb)
    if S:
        dv[:S] += (ps.transpose(1, 2) @ db).sum(0)
        dss = ps * (db @ vs.T - delta)
        dq = dq + dss @ ks
        dk[:S] += (dss.transpose(1, 2) @ qb).sum(0)
    return out + [back(dq * scale).to(torch.bfloat16), (dk * scale).to(torch.bfloat16), dv.to(torch.bfloat16)]


def _plain(s):
    c = s["case"]
    if c["op"] == "window":
        g = c["H"] // c["Hkv"]
        got = [_window_head(s["q"][:, h * g:(h + 1) * g], s["k"][:, h], s["v"][:, h],
                            s["do"][:, h * g:(h + 1) * g] if c["back"] else None, c["W"], c["S"])
               for h in range(c["Hkv"])]
        res = dict(o=torch.cat([x[0] for x in got], 1), lse=torch.cat([x[1] for x in got], 0))
        if c["back"]:
            res |= dict(dq=torch.cat([x[2] for x in got], 1), dk=torch.stack([x[3] for x in got], 1),
                        dv=torch.stack([x[4] for x in got], 1))
        return res
    cos, sin = _angles(s)
    if c["op"] == "rope":
        if c["back"]:
            sin = -sin
        return dict(q=_turn(s["q"].float(), cos, sin, c).to(torch.bfloat16),
                    k=_turn(s["k"].float(), cos, sin, c).to(torch.bfloat16))
    if not c["back"]:
        return dict(q=_norm_forward(s["q"], s["wq"], cos, sin, c), k=_norm_forward(s["k"], s["wk"], cos, sin, c))
    dq, dwq = _norm_backward(s["q"], s["wq"], s["dq"], cos, sin, c)
    dk, dwk = _norm_backward(s["k"], s["wk"], s["dk"], cos, sin, c)
    return dict(dq=dq, dk=dk, dwq=dwq, dwk=dwk)


# ------------------------------------------------------------ the library's

def _own(s):
    from headwise_chunked_context_gb300 import upipe
    c = s["case"]
    if c["op"] == "window":
        o, lse = upipe.window_forward(s["cfg"], s["q"], s["k"], s["v"])
        if not c["back"]:
            return dict(o=o, lse=lse)
        dq, dk, dv = upipe.window_backward(s["cfg"], s["q"], s["k"], s["v"], o, lse, s["do"])
        return dict(o=o, lse=lse, dq=dq, dk=dk, dv=dv)
    at = dict(pos0=c["pos0"]) if s["positions"] is None else dict(positions=s["positions"])
    if c["op"] == "rope":
        q, k = (upipe.rope_backward if c["back"] else upipe.rope_forward)(s["rope"], s["q"], s["k"], **at)
        return dict(q=q, k=k)
    if not c["back"]:
        q, k = upipe.qk_norm_rope_forward(s["rope"], s["q"], s["k"], s["wq"], s["wk"], eps=1e-6, **at)
        return dict(q=q, k=k)
    dq, dk, dwq, dwk = upipe.qk_norm_rope_backward(s["rope"], s["q"], s["k"], s["wq"], s["wk"], s["dq"], s["dk"],
                                                   eps=1e-6, **at)
    return dict(dq=dq, dk=dk, dwq=dwq, dwk=dwk)


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------- definition

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "window":
        return _exact_window(case, s)
    f = s["freqs"]
    p = s["positions"].double() if s["positions"] is not None else \
        torch.arange(case["L"], device=DEV, dtype=torch.float64) + case["pos0"]
    unit = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), p[:, None] * f)[:, None]

    def turn(x, u):  # pairs as complex numbers
        r = case["rot"]
        t, rest = x[..., :r], x[..., r:]
        if case["layout"] == "half":
            z = torch.complex(t[..., :r // 2].contiguous(), t[..., r // 2:].contiguous()) * u
            return torch.cat([z.real, z.imag, rest], -1)
        z = torch.view_as_complex(t.reshape(*t.shape[:-1], r // 2, 2).contiguous()) * u
        return torch.cat([torch.view_as_real(z).reshape(t.shape), rest], -1)

    if case["op"] == "rope":
        u = unit.conj() if case["back"] else unit
        return dict(q=turn(s["q"].double(), u), k=turn(s["k"].double(), u))
    res = {}
    for n in ("q", "k"):
        x, w = s[n].double(), s["w" + n].double()
        if case["back"]:
            x.requires_grad_(True)
            w.requires_grad_(True)
        y = turn(x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w, unit)
        if case["back"]:
            res["d" + n], res["dw" + n] = torch.autograd.grad(y, (x, w), s["d" + n].double())
        else:
            res[n] = y
    return res


def _exact_window(case, s):
    L, H, Hkv, W, S = (case[n] for n in ("L", "H", "Hkv", "W", "S"))
    g, d, B = H // Hkv, 128, 512
    heads = lambda x, n: x.double().view(L, Hkv, n, d).permute(1, 2, 0, 3)  # noqa: E731
    q, k, v = heads(s["q"], g), heads(s["k"], 1), heads(s["v"], 1)
    o, lse = torch.empty_like(q), torch.empty(Hkv, g, L, dtype=torch.float64, device=DEV)
    back = case["back"]
    if back:
        do = heads(s["do"], g)
        dq, dk, dv = torch.empty_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for a in range(0, L, B):
        e, lo = min(L, a + B), max(0, a - W + 1)
        at = torch.cat([torch.arange(min(S, lo), device=DEV), torch.arange(lo, e, device=DEV)])
        i = torch.arange(a, e, device=DEV)[:, None]
        seen = (at <= i) & ((i - at < W) | (at < S))
        t = [q[:, :, a:e], k[:, :, at], v[:, :, at]]
        if back:
            t = [x.detach().requires_grad_(True) for x in t]
        sc = (t[0] @ t[1].transpose(-1, -2) / math.sqrt(d)).masked_fill(~seen, -math.inf)
        y = torch.softmax(sc, -1) @ t[2]
        lse[:, :, a:e] = torch.logsumexp(sc.detach(), -1)
        o[:, :, a:e] = y.detach()
        if back:
            gr = torch.autograd.grad(y, t, do[:, :, a:e])
            dq[:, :, a:e] = gr[0]
            dk[:, :, at] += gr[1]
            dv[:, :, at] += gr[2]
        del t, sc, y
    flat = lambda x: x.permute(2, 0, 1, 3).reshape(L, -1, d)  # noqa: E731
    res = dict(o=flat(o), lse=lse.reshape(H, L))
    if back:
        res |= dict(dq=flat(dq), dk=flat(dk), dv=flat(dv))
    return res
