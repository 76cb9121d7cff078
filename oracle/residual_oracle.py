"""fp64 oracle of what carries the residual stream between the sublayers:
token embedding and its gradient, dropout from a counter-based generator, and
layer or RMS norm over the model width with the residual sum before it.

Plain definitions in NumPy, no code shared with the CUDA path.  Test
infrastructure only.

Embedding: y_i = scale W[t_i]; zeros for a negative token, NaN for one >= V,
neither with a gradient.
Dropout: element e (row-major, counted from `first`) is kept iff word e % 4 of
Philox 4x32-10 (Salmon et al., 2011) with counter (e // 4, call) under the key
`seed` is at least p 2^32 (p in whole steps of 2^-32), and then divided by 1 - p.
Norm: n = (s - m) / sqrt(mean((s - m)^2) + eps), y = w n + b, m = mean(s) or 0.
"""

from __future__ import annotations

import numpy as np

from oracle.upipe_oracle import bf16_round

M64 = (1 << 64) - 1


def philox(counter, key):
    """counter: four uint32 arrays (or numbers), key: two numbers; the four
    words as uint64 arrays below 2^32."""
    c = [np.asarray(w, dtype=np.uint64) for w in counter]
    low = np.uint64(0xFFFFFFFF)
    k = list(key)
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]),
             a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def steps_of(p):
    return int(p * 4294967296.0 + 0.5)


def keep(L, D, p, seed=0, call=0, first=0):
    """[L, D] truth values."""
    e = np.array([first & M64], dtype=np.uint64) + np.arange(L * D, dtype=np.uint64)
    block, low = e >> np.uint64(2), np.uint64(0xFFFFFFFF)
    call &= M64
    words = philox([block & low, block >> np.uint64(32), np.full_like(e, call & 0xFFFFFFFF), np.full_like(e, call >> 32)],
                   (seed & 0xFFFFFFFF, seed >> 32))
    return (np.choose((e & np.uint64(3)).astype(np.int64), words) >= np.uint64(steps_of(p))).reshape(L, D)


def drop(x, p, seed=0, call=0, first=0):
    x = np.asarray(x, dtype=np.float64)
    return np.where(keep(*x.shape, p, seed, call, first), x / (1 - steps_of(p) / 4294967296.0), 0.0)


def add(x, res=None, **mask):
    """res + drop(x), not rounded; no mask: their sum."""
    x = np.asarray(x, dtype=np.float64)
    y = drop(x, **mask) if mask else x
    return y if res is None else res + y


def stats(s, eps, rms):
    """(mean or 0, 1 / sqrt(spread + eps)) of each row, [L, 1]."""
    m = np.zeros((s.shape[0], 1)) if rms else s.mean(-1, keepdims=True)
    return m, 1 / np.sqrt(np.mean((s - m) ** 2, -1, keepdims=True) + eps)


def norm(s, w, b, eps, rms):
    s = np.asarray(s, dtype=np.float64)
    m, r = stats(s, eps, rms)
    return (s - m) * r * w + (0 if b is None else b)


def norm_bwd(s, w, dy, ds, eps, rms):
    """(gradient of s, dw, db); the gradient of x is the first behind the mask."""
    s = np.asarray(s, dtype=np.float64)
    m, r = stats(s, eps, rms)
    n, g = (s - m) * r, dy * w
    d = r * (g - (0 if rms else g.mean(-1, keepdims=True)) - n * np.mean(g * n, -1, keepdims=True))
    return d if ds is None else d + ds, (dy * n).sum(0), dy.sum(0)


def embed(tokens, W, scale=1.0):
    t = np.asarray(tokens)
    y = np.zeros((len(t), W.shape[1]))
    real = (t >= 0) & (t < W.shape[0])
    y[real] = scale * W[t[real]]
    y[t >= W.shape[0]] = np.nan
    return y


def embed_bwd(tokens, dy, V, scale=1.0):
    """(dW, the sizes of its terms added up, terms per row)."""
    t = np.asarray(tokens)
    real = (t >= 0) & (t < V)
    dW, size, count = np.zeros((V, dy.shape[1])), np.zeros((V, dy.shape[1])), np.zeros(V, dtype=np.int64)
    np.add.at(dW, t[real], scale * dy[real])
    np.add.at(size, t[real], np.abs(scale * dy[real]))
    np.add.at(count, t[real], 1)
    return dW, size, count


__all__ = ["philox", "keep", "drop", "add", "stats", "norm", "norm_bwd", "embed", "embed_bwd", "bf16_round"]
