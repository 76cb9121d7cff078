"""fp64 oracle of what stands around the attention core: rotary positions,
norms of queries and keys with the rotation, and causal attention with a
sliding window and sink tokens.

Plain definitions in NumPy fp64, one loop per head, no code shared with the
CUDA path.  Test infrastructure only.

Rotary positions: y_a = c (x_a cos(p f_i) - x_b sin(p f_i)), y_b = c (x_a
sin(p f_i) + x_b cos(p f_i)) for (a, b) = (i, i + rot/2) ("half") or (2i,
2i + 1) ("interleaved"); elements from rot on pass through.
Norm: n = x / sqrt(mean(x^2) + eps), z = w n, then the rotation.
Window: key j is visible to query i iff j <= i and (i - j < W or j < S).
"""

from __future__ import annotations

import numpy as np

from oracle.upipe_oracle import bf16_round


def pairs(rot, layout):
    i = np.arange(rot // 2)
    return (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)


def frequencies(rot, theta=500000.0, scaling=None):
    """theta^(-2i/rot); ("linear", factor) divides by factor; ("bands",
    factor, low, high, orig_len) blends between kept (at least `high` turns
    in orig_len positions) and divided (at most `low`)."""
    f = np.array([theta ** (-2.0 * i / rot) for i in range(rot // 2)])
    if scaling and scaling[0] == "linear":
        f = f / scaling[1]
    if scaling and scaling[0] == "bands":
        _, factor, low, high, orig = scaling
        turns = orig * f / (2 * np.pi)
        keep = np.clip((turns - low) / (high - low), 0.0, 1.0)
        f = f * (keep + (1 - keep) / factor)
    return f


def rope(x, positions, freqs, rot, layout, magnitude=1.0, transpose=False):
    """x [L, heads, d] fp64, positions [L]."""
    x = np.asarray(x, dtype=np.float64)
    a, b = pairs(rot, layout)
    ang = np.asarray(positions, dtype=np.float64)[:, None] * freqs[None, :]
    c, s = magnitude * np.cos(ang)[:, None], magnitude * np.sin(ang)[:, None]
    if transpose:
        s = -s
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    return y


def norm_rope(x, w, eps, positions, freqs, rot, layout, magnitude=1.0):
    x = np.asarray(x, dtype=np.float64)
    n = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    return rope(n * w, positions, freqs, rot, layout, magnitude)


def norm_rope_bwd(x, w, eps, dy, positions, freqs, rot, layout, magnitude=1.0):
    """(dx, dw) and the sum of the absolute terms of dw, the scale of its
    rounding errors."""
    x = np.asarray(x, dtype=np.float64)
    r = 1.0 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    n = x * r
    dz = rope(dy, positions, freqs, rot, layout, magnitude, transpose=True)
    dn = dz * w
    dx = r * (dn - n * np.mean(dn * n, -1, keepdims=True))
    return dx, np.sum(dz * n, (0, 1)), np.sum(np.abs(dz * n), (0, 1))


def visible(i, j, window, sinks):
    """Mask of queries i (rows) and keys j (columns)."""
    i, j = np.asarray(i)[:, None], np.asarray(j)[None, :]
    return (j <= i) & ((i - j < window) | (j < sinks))


def _probs(q, k, window, sinks):
    L, d = q.shape
    s = q @ k.T / np.sqrt(d)
    s[~visible(np.arange(L), np.arange(L), window, sinks)] = -np.inf
    m = s.max(1, keepdims=True)
    lse = m[:, 0] + np.log(np.exp(s - m).sum(1))
    return np.exp(s - lse[:, None]), lse


def window_fwd(q, k, v, window, sinks):
    """q [L, H, d], k, v [L, Hkv, d] -> o [L, H, d], lse [H, L]."""
    L, H, d = q.shape
    g = H // k.shape[1]
    o, lse = np.empty((L, H, d)), np.empty((H, L))
    for h in range(H):
        p, lse[h] = _probs(q[:, h], k[:, h // g], window, sinks)
        o[:, h] = p @ v[:, h // g]
    return o, lse


def window_bwd(q, k, v, o, do, window, sinks, bf16_operands=False):
    """dq, dk, dv.  bf16_operands: P and dS enter their products rounded to
    bf16 (every contraction input in bf16, all else exact)."""
    L, H, d = q.shape
    g = H // k.shape[1]
    rnd = bf16_round if bf16_operands else (lambda x: x)
    dq, dk, dv = np.zeros((L, H, d)), np.zeros(k.shape), np.zeros(v.shape)
    for h in range(H):
        kv = h // g
        p, _ = _probs(q[:, h], k[:, kv], window, sinks)
        dp = do[:, h] @ v[:, kv].T
        delta = np.sum(do[:, h] * o[:, h], 1, keepdims=True)
        ds = rnd(p * (dp - delta))
        dq[:, h] = ds @ k[:, kv] / np.sqrt(d)
        dk[:, kv] += ds.T @ q[:, h] / np.sqrt(d)
        dv[:, kv] += rnd(p).T @ do[:, h]
    return dq, dk, dv
