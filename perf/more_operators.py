"""Cases of the operators that carry the residual stream between the layers:
token embedding and its gradient by sorted tokens, layer and RMS norm over the
model width with the residual sum and dropout before it, and dropout from a
counter-based generator.

Where ``own`` is false, ``run`` computes them in plain torch operations in 32
bits (random bits in 64-bit integers); where it is true, ``run`` calls the
library.
"""

import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5
M32 = (1 << 32) - 1


# ------------------------------------------------------------------- cases

def listed():
    return [
        # The next token of a sequence: launch latency is all there is.
        dict(name="embed one token", op="embed", back=False, L=1, V=128256, D=4096, table="fp32", ids="int64", pad=0),
        # The 32B-shaped model's tokens at the full context, from the fp32 master table.
        dict(name="embed forward", op="embed", back=False, L=131072, V=152064, D=5120, table="fp32", ids="int32",
             pad=0),
        # The 8B-shaped model's table gradient: almost all of its rows are zeros.
        dict(name="embed gradient", op="embed", back=True, L=32768, V=128256, D=4096, table="fp32", ids="int32", pad=0),
        # A short padded batch of a small model: gradient of an odd number of rows.
        dict(name="embed ragged gradient", op="embed", back=True, L=4099, V=30011, D=1032, table="bf16", ids="int64",
             pad=513),
        # One token between two sublayers: residual sum and RMS norm.
        dict(name="norm one token", op="norm", back=False, L=1, D=5120, rms=True, bias=False, res=True, p=0.0,
             wide=False),
        # A block's first norm at the 8B shape, no residual.
        dict(name="norm forward", op="norm", back=False, L=32768, D=4096, rms=False, bias=True, res=False, p=0.0,
             wide=False),
        # Its gradients with the weight's and the bias's.
        dict(name="norm backward", op="norm", back=True, L=32768, D=4096, rms=False, bias=True, res=False, p=0.0,
             wide=False),
        # Between two sublayers of the 32B-shaped model at the full context: dropout, residual sum, RMS norm.
        dict(name="add norm forward", op="norm", back=False, L=131072, D=5120, rms=True, bias=False, res=True, p=0.1,
             wide=False),
        # Its gradients, the residual path's gradient added.
        dict(name="add norm backward", op="norm", back=True, L=131072, D=5120, rms=True, bias=False, res=True, p=0.1,
             wide=False),
        # A short ragged batch, rows inside a wider buffer, a width that no power of two divides much.
        dict(name="norm ragged backward", op="norm", back=True, L=1025, D=1032, rms=False, bias=True, res=True, p=0.0,
             wide=True),
        # A sublayer's output joins the residual stream, no norm behind it (the last block of a stage).
        dict(name="dropout add", op="drop", back=False, L=131072, D=5120, res=True, p=0.1, wide=False),
        # The gradient of a small ragged one.
        dict(name="dropout ragged gradient", op="drop", back=True, L=333, D=1000, res=False, p=0.5, wide=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    most = 10 * 131072 * 5120  # bytes of the dearest listed case
    op = rng.choice(["embed", "norm", "norm", "drop"])
    while True:
        L, D = _log(rng, 1, 131072), 8 * _log(rng, 8, 2048)
        if op == "embed":
            V, back = _log(rng, 256, 152064), rng.random() < 0.6
            c = dict(op=op, back=back, L=L, V=V, D=D, table=rng.choice(["fp32", "bf16"]),
                     ids=rng.choice(["int32", "int64"]), pad=rng.choice([0, 0, rng.randint(0, L)]))
            if D <= 8192 and V * D * 4 + L * D * 6 <= most:
                return c
        else:
            res = rng.random() < 0.6
            c = dict(op=op, back=rng.random() < 0.5, L=L, D=D)
            if op == "norm":
                c |= dict(rms=rng.random() < 0.5, bias=rng.random() < 0.5)
            c |= dict(res=res, p=rng.choice([0.0, 0.1, rng.uniform(0.01, 0.9)]) if res or op == "drop" else 0.0,
                      wide=rng.random() < 0.3)
            if op == "drop":
                c["p"] = c["p"] or 0.2
            if 10 * L * D <= most:
                return c


def _share(V):
    """Chance of each token: falls with its index, as a tokenizer's ids do."""
    at = torch.arange(V, dtype=torch.float64)
    return torch.log((at + 2) / (at + 1)) / math.log(V + 1)


def work(case):
    L, D, back = case["L"], case["D"], case["back"]
    e = L * D
    if case["op"] == "embed":
        V, n = case["V"], L - case["pad"]
        tok = L * (8 if case["ids"] == "int64" else 4)
        if back:
            return dict(bytes=4 * V * D + 2 * n * D + tok, flops=n * D)
        rows = float((1 - (1 - _share(V)) ** n).sum())  # expected distinct tokens
        return dict(bytes=int(rows * D * (4 if case["table"] == "fp32" else 2)) + 2 * e + tok, flops=n * D)
    drop = 2 if case["p"] else 0
    if case["op"] == "drop":
        return dict(bytes=(4 if back or not case["res"] else 6) * e, flops=(drop + 1) * e)
    w = 4 * D * (2 if case["bias"] else 1)
    if not back:
        return dict(bytes=(8 if case["res"] else 4) * e + w, flops=(8 + drop) * e)
    b = 6 + (2 if case["res"] else 0) + (2 if case["p"] else 0)  # s, dy, dx, and ds, and dx behind the mask
    return dict(bytes=b * e + 4 * D + w, flops=(16 + drop) * e)


# ------------------------------------------------------------------- inputs

def _rows(case, g, *, scale=None, std=1.0):
    """[L, D] bf16, a slice of wider rows where the case says so."""
    L, D = case["L"], case["D"]
    x = torch.randn(L, D, generator=g, device=DEV) * std
    if scale is not None:
        x *= scale
    x = x.to(torch.bfloat16)
    if not case["wide"]:
        return x
    buf = torch.zeros(L, D + 72, dtype=torch.bfloat16, device=DEV)
    buf[:, 8:8 + D] = x
    return buf[:, 8:8 + D]


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    L, D = case["L"], case["D"]
    s = dict(case=case)
    if case["op"] == "embed":
        V = case["V"]
        u = torch.rand(L, generator=g, device=DEV, dtype=torch.float64)
        t = (torch.exp(u * math.log(V + 1)) - 1).long().clamp_(0, V - 1)
        if case["pad"]:
            t[L - case["pad"]:] = -1
        s["tokens"] = t.to(torch.int32 if case["ids"] == "int32" else torch.int64)
        s["scale"] = math.sqrt(D)
        if case["back"]:
            s["dy"] = torch.randn(L, D, generator=g, device=DEV).to(torch.bfloat16)
        else:
            s["W"] = torch.randn(V, D, generator=g, device=DEV) * 0.02
            if case["table"] == "bf16":
                s["W"] = s["W"].to(torch.bfloat16)
        return s
    # a mask's key is a seed and the number of the call within the run
    s["p"], s["seed"], s["call"] = case["p"], (seed * 0x9E3779B97F4A7C15 + 12345) & ((1 << 64) - 1), (7 << 32) + L
    if case["op"] == "drop":
        s["x"] = _rows(case, g)
        s["res"] = _rows(case, g, std=3.0) if case["res"] else None
    else:
        s["w"] = 1.0 + 0.2 * torch.randn(D, generator=g, device=DEV)
        s["b"] = 0.1 * torch.randn(D, generator=g, device=DEV) if case["bias"] else None
        # a residual stream: channels of unlike size, a few of them far above the rest
        scale = torch.exp(0.5 * torch.randn(D, generator=g, device=DEV))
        scale[:: max(1, D // 4)] *= 30.0
        if case["back"]:
            s["s"], s["dy"] = _rows(case, g, scale=scale), _rows(case, g)
            s["ds"] = _rows(case, g) if case["res"] else None
        else:
            s["x"] = _rows(case, g, scale=None if case["res"] else scale)
            s["res"] = _rows(case, g, scale=scale) if case["res"] else None
    if own:
        from headwise_chunked_context_gb300 import upipe
        s["drop"] = upipe.Dropout(case["p"], seed=s["seed"], call=s["call"]) if case["p"] else None
    return s


# --------------------------------------------------------------- plain form

def _plain_keep(s):
    """Which elements stay, [L, D], and the factor of those that do.  Philox
    4x32-10 (Salmon et al., 2011): word e % 4 of the block of counter
    (e // 4, call) under the key `seed` is element e's."""
    L, D = s["case"]["L"], s["case"]["D"]
    at = torch.arange(L * D // 4, device=DEV)
    c0, c1 = at & M32, at >> 32
    c2, c3 = torch.full_like(at, s["call"] & M32), torch.full_like(at, s["call"] >> 32)
    k0, k1 = s["seed"] & M32, s["seed"] >> 32
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # modulo 2^64, which holds both words
        c0, c1, c2, c3 = ((b >> 32) & M32) ^ c1 ^ k0, b & M32, ((a >> 32) & M32) ^ c3 ^ k1, a & M32
        k0, k1 = (k0 + 0x9E3779B9) & M32, (k1 + 0xBB67AE85) & M32
    cut = round(s["p"] * 2.0 ** 32)
    keep = torch.stack([c0 >= cut, c1 >= cut, c2 >= cut, c3 >= cut], 1).view(L, D)
    return keep, 2.0 ** 32 / (2.0 ** 32 - cut)


def _dropped(x, s):
    """x [L, D] fp32 behind the mask."""
    if not s["p"]:
        return x
    keep, factor = _plain_keep(s)
    return torch.where(keep, x * factor, 0.0)


def _plain(s):
    c = s["case"]
    if c["op"] == "embed":
        if not c["back"]:
            t = s["tokens"].long()
            y = s["W"][t.clamp(min=0)].float() * s["scale"]
            return dict(y=torch.where(t[:, None] >= 0, y, 0.0).to(torch.bfloat16))
        t = s["tokens"].long()
        dW = torch.zeros(c["V"] + 1, c["D"], device=DEV)
        dW.index_add_(0, torch.where(t >= 0, t, c["V"]), s["dy"].float())
        return dict(dW=(dW[:c["V"]] * s["scale"]))
    if c["op"] == "drop":
        y = _dropped(s["x"].float(), s)
        return dict(y=(y if s["res"] is None else s["res"].float() + y).to(torch.bfloat16))
    if not c["back"]:
        out = {}
        x = s["x"]
        if c["res"]:
            x = out["s"] = (s["res"].float() + _dropped(x.float(), s)).to(torch.bfloat16)
        x = x.float()
        if not c["rms"]:
            x = x - x.mean(-1, keepdim=True)
        y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s["w"]
        return out | dict(y=(y if s["b"] is None else y + s["b"]).to(torch.bfloat16))
    x, dy = s["s"].float(), s["dy"].float()
    if not c["rms"]:
        x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    n, g = x * r, dy * s["w"]
    out = dict(dw=(dy * n).sum(0))
    if c["bias"]:
        out["db"] = dy.sum(0)
    d = g - n * (g * n).mean(-1, keepdim=True)
    if not c["rms"]:
        d = d - g.mean(-1, keepdim=True)
    d = d * r
    if c["res"]:
        d = d + s["ds"].float()
    out["dres" if c["p"] else "dx"] = d.to(torch.bfloat16)
    if c["p"]:
        out["dx"] = _dropped(d, s).to(torch.bfloat16)
    return out


# ------------------------------------------------------------ the library's

def _own(s):
    from headwise_chunked_context_gb300 import upipe
    c = s["case"]
    if c["op"] == "embed":
        if not c["back"]:
            return dict(y=upipe.embed_forward(s["tokens"], s["W"], scale=s["scale"]))
        return dict(dW=upipe.embed_backward(s["tokens"], s["dy"], c["V"], scale=s["scale"]))
    if c["op"] == "drop":
        if c["back"] and not c["res"]:
            return dict(y=upipe.dropout_backward(s["drop"], s["x"]))
        return dict(y=upipe.dropout_forward(s["drop"], s["x"], s["res"]))  # or onto another gradient
    if not c["back"]:
        y, total = upipe.layer_norm_forward(s["x"], s["w"], s["b"], eps=EPS, rms=c["rms"], residual=s["res"],
                                            dropout=s["drop"])
        return dict(s=total, y=y) if c["res"] else dict(y=y)
    dx, dres, dw, db = upipe.layer_norm_backward(s["s"], s["w"], s["dy"], s["ds"], eps=EPS, rms=c["rms"],
                                                 bias=c["bias"], dropout=s["drop"])
    out = dict(dw=dw)
    if c["bias"]:
        out["db"] = db
    out["dres" if c["p"] else "dx"] = dres
    if c["p"]:
        out["dx"] = dx
    return out


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------- definition

def _philox_block(counter, key):
    """Four words of counter words `counter` under key words `key`; products
    by halves of 16 bits, so that nothing leaves 63."""
    def high_low(a, m):
        low, high = a * (m & 0xFFFF), a * (m >> 16)
        mid = high + (low >> 16)
        return mid >> 16, ((mid & 0xFFFF) << 16) | (low & 0xFFFF)

    x = list(counter)
    for r in range(10):
        ka, kb = (key[0] + r * 0x9E3779B9) & M32, (key[1] + r * 0xBB67AE85) & M32
        ha, la = high_low(x[0], 0xD2511F53)
        hb, lb = high_low(x[2], 0xCD9E8D57)
        x = [hb.bitwise_xor(x[1]).bitwise_xor(ka), lb, ha.bitwise_xor(x[3]).bitwise_xor(kb), la]
    return x


def _mask(s, lo, hi):
    """Factors of rows lo .. hi: 0 or 1 / (1 - p), p in whole steps of 2^-32."""
    D = s["case"]["D"]
    at = torch.arange(lo * D, hi * D, device=DEV)
    block = torch.arange(lo * D // 4, hi * D // 4, device=DEV)
    words = _philox_block([block & M32, block >> 32] +
                          [torch.full_like(block, w) for w in (s["call"] & M32, s["call"] >> 32)],
                          (s["seed"] & M32, s["seed"] >> 32))
    u = torch.stack(words, -1).reshape(-1)
    assert u.numel() == at.numel()
    steps = round(s["p"] * 4294967296)
    return ((u >= steps).double() / (1 - steps / 4294967296)).view(hi - lo, D)


def exact(case, seed):
    s = prepare(case, seed)
    L, D = case["L"], case["D"]
    if case["op"] == "embed":
        t = s["tokens"].long()
        real = t >= 0
        if not case["back"]:
            y = torch.zeros(L, D, dtype=torch.float64, device=DEV)
            y[real] = s["W"][t[real]].double() * s["scale"]
            return dict(y=y)
        dW = torch.zeros(case["V"], D, dtype=torch.float64, device=DEV)
        for a in range(0, L, 16384):
            at = slice(a, a + 16384)
            dW.index_add_(0, t[at][real[at]], s["dy"][at][real[at]].double() * s["scale"])
        return dict(dW=dW)
    step = max(1, (1 << 25) // D)
    parts = {}

    def put(name, value):
        parts.setdefault(name, []).append(value)

    dw = torch.zeros(D, dtype=torch.float64, device=DEV)
    db = torch.zeros(D, dtype=torch.float64, device=DEV)
    for lo in range(0, L, step):
        hi = min(L, lo + step)
        f = _mask(s, lo, hi) if case["p"] else torch.ones((), dtype=torch.float64, device=DEV)
        if case["op"] == "drop":
            y = s["x"][lo:hi].double() * f
            put("y", y if s["res"] is None else y + s["res"][lo:hi].double())
            continue

        def norm(x, w, b):
            v = x if case["rms"] else x - x.mean(-1, keepdim=True)
            y = v / (v.square().mean(-1, keepdim=True) + EPS).sqrt() * w
            return y if b is None else y + b

        w, b = s["w"].double(), s["b"].double() if case["bias"] else None
        if not case["back"]:
            x = s["x"][lo:hi].double()
            if case["res"]:
                x = s["res"][lo:hi].double() + x * f
                put("s", x)
                x = x.to(torch.bfloat16).double()  # the norm is of the sum as it is kept
            put("y", norm(x, w, b))
            continue
        # the gradient of sum(y dy) + sum(s ds), by differentiation
        x, w = s["s"][lo:hi].double().requires_grad_(True), w.requires_grad_(True)
        leaves = (x, w)
        if case["bias"]:
            b = b.requires_grad_(True)
            leaves += (b,)
        got = torch.autograd.grad(norm(x, w, b), leaves, s["dy"][lo:hi].double())
        d = got[0] if s["ds"] is None else got[0] + s["ds"][lo:hi].double()
        dw += got[1]
        if case["bias"]:
            db += got[2]
        put("dres" if case["p"] else "dx", d)
        if case["p"]:
            put("dx", d * f)
    out = {n: torch.cat(v) if len(v) > 1 else v[0] for n, v in parts.items()}
    if case["op"] == "norm" and case["back"]:
        out["dw"] = dw
        if case["bias"]:
            out["db"] = db
    return out
