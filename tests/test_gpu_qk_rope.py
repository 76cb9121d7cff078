"""GPU parity of rotary positions and query/key norms against the fp64 oracle.

Tolerances, element by element: an output is rounded to bf16 once, by at most
2^-8 of its size (half a step).  Before that, an angle is off by at most
pi 2^-25 (its fp32 fraction of a turn) + 2^-22 (two fp64 products of a
frequency and a position below 2^31, the oracle's and ours) and a sine or
cosine by two more units of 2^-24: under 5e-7, and 1e-6 with the products of
the rotation.  It scales with |z_a| + |z_b|.  The norm adds the relative error
of a sum of d <= 256 squares and of an inverse root: under 3e-6.  A weight's
gradient adds up at most 200 terms one after another in the tests' sizes (the
rest pairwise): 200 2^-24 = 1.2e-5 of the sum of its terms' sizes, and the
terms' own 5e-6."""

import math

import numpy as np
import pytest
import torch

from headwise_chunked_context_gb300 import upipe
from oracle import local_oracle as loc
from tests.gpu_common import ensure_lib, f64

pytestmark = pytest.mark.gpu

HALF_STEP = 2.0 ** -8
ANGLE, NORM, WEIGHT = 1e-6, 4e-6, 2e-5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def _randn(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(torch.bfloat16).cuda()


def _pair_size(x, rot, layout):
    """|z_a| + |z_b| at both members of each pair, |z| elsewhere."""
    a, b = loc.pairs(rot, layout)
    y = np.abs(x)
    y[..., a] = y[..., b] = y[..., a] + y[..., b]
    return y


def _near(got, want, slack, name):
    got = f64(got)
    assert np.all(np.isfinite(got)), name
    over = np.abs(got - want) - (HALF_STEP * np.abs(want) + slack)
    assert over.max() <= 0, f"{name}: {over.max():.3e} over at {np.unravel_index(over.argmax(), over.shape)}"


# L, H, Hkv, d, rot, layout: every path (16-byte vectors in both layouts, two-byte), lane groups of
# 1 to 16, head counts that leave lanes idle, one token and many
CASES = [
    (1, 1, 0, 128, 128, "half"), (1, 32, 8, 128, 128, "half"), (3, 5, 3, 128, 128, "interleaved"),
    (300, 6, 2, 128, 64, "half"), (300, 6, 2, 128, 64, "interleaved"), (65, 9, 3, 128, 0, "half"),
    (33, 4, 1, 128, 34, "half"), (33, 4, 1, 128, 34, "interleaved"), (40, 3, 3, 16, 16, "half"),
    (40, 40, 8, 16, 2, "interleaved"), (21, 7, 1, 8, 8, "half"), (21, 7, 1, 8, 4, "interleaved"),
    (50, 3, 2, 72, 72, "half"), (50, 3, 2, 96, 48, "half"), (50, 3, 2, 80, 80, "interleaved"),
    (19, 5, 1, 192, 96, "half"), (19, 5, 1, 256, 256, "half"), (19, 5, 1, 256, 254, "half"),
    (19, 5, 1, 256, 250, "interleaved"), (2600, 3, 1, 64, 64, "half"), (31, 3, 2, 72, 40, "interleaved"),
    (31, 3, 2, 72, 8, "half"), (31, 3, 2, 128, 8, "half"), (23, 5, 2, 248, 248, "half"), (23, 5, 2, 256, 24, "half"),
    (23, 5, 2, 248, 246, "interleaved"), (23, 3, 1, 248, 244, "half"),
]


@pytest.mark.parametrize("L,H,Hkv,d,rot,layout", CASES)
@pytest.mark.parametrize("transpose", [False, True])
def test_rope_matches_oracle(L, H, Hkv, d, rot, layout, transpose):
    q, k = _randn(0, L, H, d), _randn(1, L, Hkv, d) if Hkv else None
    r = upipe.Rope(d, rot=rot, layout=layout, magnitude=1.25)
    pos0 = 70000
    qo, ko = (upipe.rope_backward if transpose else upipe.rope_forward)(r, q, k, pos0=pos0)
    f, pos = np.array(r.freqs), np.arange(L) + pos0
    for x, y, n in ((q, qo, "q"), (k, ko, "k")):
        if x is None:
            assert y is None
            continue
        want = loc.rope(f64(x), pos, f, rot, layout, 1.25, transpose)
        _near(y, want, 1.25 * ANGLE * _pair_size(f64(x), rot, layout), n)
        assert torch.equal(y[..., rot:], x[..., rot:])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("scaling", [None, ("linear", 4.0), ("bands", 8.0, 1.0, 4.0, 8192)])
def test_rope_far_and_given_positions(layout, scaling):
    at = [0, 1, 2, 5, 1 << 20, (1 << 21) + 3, 123456789, (1 << 31) - 1, -1, -(1 << 31), 17]
    pos = torch.tensor(at, dtype=torch.int32, device="cuda")
    q, k = _randn(2, len(at), 4, 128), _randn(3, len(at), 2, 128)
    r = upipe.Rope(128, layout=layout, scaling=scaling)
    qo, ko = upipe.rope_forward(r, q, k, positions=pos)
    for x, y in ((q, qo), (k, ko)):
        want = loc.rope(f64(x), at, np.array(r.freqs), 128, layout)
        _near(y, want, ANGLE * _pair_size(f64(x), 128, layout), "far")
    # pos0 is the same positions
    one = upipe.rope_forward(r, q[5:6], k[5:6], pos0=(1 << 21) + 3)
    assert torch.equal(one[0], qo[5:6]) and torch.equal(one[1], ko[5:6])


def test_rope_beyond_31_bits_by_pos0():
    """pos0 past 2^31: the turns are still exact (the oracle's angle, in fp64,
    is off by 2^40 2^-53 of a frequency of 1, and ours as much)."""
    q = _randn(4, 2, 3, 128)
    r = upipe.Rope(128)
    y, _ = upipe.rope_forward(r, q, pos0=1 << 40)
    want = loc.rope(f64(q), [1 << 40, (1 << 40) + 1], np.array(r.freqs), 128, "half")
    _near(y, want, (ANGLE + 2 * 2.0 ** -12) * _pair_size(f64(q), 128, "half"), "2^40")


@pytest.mark.parametrize("L,H,Hkv,d,rot,layout", CASES)
def test_norm_rope_matches_oracle(L, H, Hkv, d, rot, layout):
    q, k = _randn(0, L, H, d), _randn(1, L, Hkv, d) if Hkv else None
    dq, dk = _randn(5, L, H, d), _randn(6, L, Hkv, d) if Hkv else None
    g = torch.Generator().manual_seed(7)
    wq, wk = (1 + 0.2 * torch.randn(2, d, generator=g)).cuda().unbind(0)
    wq, wk = wq.clone(), wk.clone()
    r = upipe.Rope(d, rot=rot, layout=layout, magnitude=0.75)
    pos0, eps = 1234, 1e-5
    pos, f = np.arange(L) + pos0, np.array(r.freqs)
    kw = dict(eps=eps, pos0=pos0)
    qo, ko = upipe.qk_norm_rope_forward(r, q, k, wq, wk, **kw)
    gq, gk, gwq, gwk = upipe.qk_norm_rope_backward(r, q, k, wq, wk, dq, dk, **kw)
    for x, w, y, dy, dx, dw, n in ((q, wq, qo, dq, gq, gwq, "q"), (k, wk, ko, dk, gk, gwk, "k")):
        if x is None:
            assert y is None and dx is None and dw is None
            continue
        x, w, dy = f64(x), f64(w), f64(dy)
        z = loc.norm_rope(x, w, eps, pos, np.zeros(rot // 2), rot, layout)  # unrotated
        _near(y, loc.norm_rope(x, w, eps, pos, f, rot, layout, 0.75),
              0.75 * (ANGLE + NORM) * _pair_size(z, rot, layout), n)
        want, want_w, size_w = loc.norm_rope_bwd(x, w, eps, dy, pos, f, rot, layout, 0.75)
        rr = 1 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
        dn = np.abs(w) * 0.75 * _pair_size(dy, rot, layout)
        _near(dx, want, NORM * rr * (dn + np.abs(x) * rr * np.mean(dn * np.abs(x) * rr, -1, keepdims=True)), "d" + n)
        assert np.all(np.abs(f64(dw) - want_w) <= WEIGHT * (size_w + np.sum(_pair_size(dy, rot, layout) * np.abs(x) * rr,
                                                                           (0, 1)))), "dw" + n


def _fused(seed, L, H, Hkv, d):
    return _randn(seed, L, H + 2 * Hkv, d)


@pytest.mark.parametrize("d,rot", [(128, 128), (72, 40)])
def test_strided_and_in_place_calls_give_the_dense_calls_bits(d, rot):
    L, H, Hkv = 77, 6, 2
    qkv = _fused(8, L, H, Hkv, d)
    q, k = qkv[:, :H], qkv[:, H:H + Hkv]
    w = torch.linspace(0.5, 1.5, d, device="cuda")
    r = upipe.Rope(d, rot=rot)
    want = upipe.rope_forward(r, q.contiguous(), k.contiguous(), pos0=5)
    got = upipe.rope_forward(r, q, k, pos0=5)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # head-major output
    hm = torch.full((H + Hkv, L, d), 7.0, dtype=torch.bfloat16, device="cuda")
    upipe.rope_apply(r, q, k, hm[:H].transpose(0, 1), hm[H:].transpose(0, 1), pos0=5)
    assert torch.equal(hm[:H].transpose(0, 1), want[0]) and torch.equal(hm[H:].transpose(0, 1), want[1])
    # in place, inside the fused buffer: the values stay as they were
    buf = qkv.clone()
    upipe.rope_apply(r, buf[:, :H], buf[:, H:H + Hkv], buf[:, :H], buf[:, H:H + Hkv], pos0=5)
    assert torch.equal(buf[:, :H], want[0]) and torch.equal(buf[:, H:H + Hkv], want[1])
    assert torch.equal(buf[:, H + Hkv:], qkv[:, H + Hkv:])
    # norm: strided and in place, forward and backward
    nw = upipe.qk_norm_rope_forward(r, q.contiguous(), k.contiguous(), w, w)
    buf = qkv.clone()
    upipe.qk_norm_rope_fwd(r, buf[:, :H], buf[:, H:H + Hkv], w, w, buf[:, :H], buf[:, H:H + Hkv])
    assert torch.equal(buf[:, :H], nw[0]) and torch.equal(buf[:, H:H + Hkv], nw[1])
    dqkv = _fused(9, L, H, Hkv, d)
    dq, dk = dqkv[:, :H], dqkv[:, H:H + Hkv]
    bw = upipe.qk_norm_rope_backward(r, q.contiguous(), k.contiguous(), w, w, dq.contiguous(), dk.contiguous())
    dwq, dwk = torch.empty_like(w), torch.empty_like(w)
    buf = dqkv.clone()
    dq, dk = buf[:, :H], buf[:, H:H + Hkv]
    upipe.qk_norm_rope_bwd(r, q, k, w, w, dq, dk, dq, dk, dwq, dwk)
    for a, b in zip((dq, dk, dwq, dwk), bw):
        assert torch.equal(a, b)
    assert torch.equal(buf[:, H + Hkv:], dqkv[:, H + Hkv:])


def test_broadcast_input_rows():
    """One row for all tokens (stride 0): read as it stands."""
    x = _randn(10, 1, 4, 128)
    r = upipe.Rope(128)
    y, _ = upipe.rope_forward(r, x.expand(9, 4, 128))
    assert torch.equal(y, upipe.rope_forward(r, x.repeat(9, 1, 1))[0])


def test_more_tokens_than_resident_warps_and_the_same_bits_again():
    L, H, Hkv = 20001, 4, 1
    q, k, dq, dk = _randn(11, L, H, 128), _randn(12, L, Hkv, 128), _randn(13, L, H, 128), _randn(14, L, Hkv, 128)
    w = torch.ones(128, device="cuda")
    r = upipe.Rope(128)
    a = upipe.qk_norm_rope_backward(r, q, k, w, w, dq, dk)
    b = upipe.qk_norm_rope_backward(r, q, k, w, w, dq, dk)
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    f, pos = np.array(r.freqs), np.arange(L)
    for x, dy, dw in ((q, dq, a[2]), (k, dk, a[3])):
        _, want, size = loc.norm_rope_bwd(f64(x), np.ones(128), 1e-6, f64(dy), pos, f, 128, "half")
        assert np.all(np.abs(f64(dw) - want) <= WEIGHT * 2 * size)


def test_zero_and_huge_heads():
    """A head of zeros stays zero (eps > 0); values near bf16's largest square
    past fp32 and follow the formula there: the norm is infinite, n is 0."""
    q = torch.zeros(2, 3, 128, dtype=torch.bfloat16, device="cuda")
    q[1] = 1e30
    w = torch.ones(128, device="cuda")
    r = upipe.Rope(128)
    y, _ = upipe.qk_norm_rope_forward(r, q, None, w, None)
    assert torch.equal(y, torch.zeros_like(y))
    q[:] = float("nan")
    y, _ = upipe.qk_norm_rope_forward(r, q, None, w, None)
    assert torch.isnan(y).all()


def test_on_another_stream_and_captured():
    L, H, Hkv = 130, 4, 2
    q, k, dq, dk = _randn(15, L, H, 128), _randn(16, L, Hkv, 128), _randn(17, L, H, 128), _randn(18, L, Hkv, 128)
    w = torch.linspace(0.5, 1.5, 128, device="cuda")
    r = upipe.Rope(128)
    want = upipe.qk_norm_rope_forward(r, q, k, w, w), upipe.qk_norm_rope_backward(r, q, k, w, w, dq, dk)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    out = [torch.empty_like(t) for t in (q, k, q, k, w, w)]
    upipe.qk_norm_rope_fwd(r, q, k, w, w, out[0], out[1], stream=st)
    upipe.qk_norm_rope_bwd(r, q, k, w, w, dq, dk, *out[2:], stream=st)
    st.synchronize()
    for a, b in zip(out, want[0] + want[1]):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f = upipe.qk_norm_rope_forward(r, q, k, w, w)
        b = upipe.qk_norm_rope_backward(r, q, k, w, w, dq, dk)
    q.copy_(_randn(19, L, H, 128))
    graph.replay()
    torch.cuda.synchronize()
    want = upipe.qk_norm_rope_forward(r, q, k, w, w), upipe.qk_norm_rope_backward(r, q, k, w, w, dq, dk)
    for x, y in zip(f + b, want[0] + want[1]):
        assert torch.equal(x, y)


def test_workspace_refusals():
    q = _randn(20, 8, 2, 128)
    w = torch.ones(128, device="cuda")
    r = upipe.Rope(128)
    need = upipe.qk_norm_rope_workspace_bytes(r, 8, 2)
    with pytest.raises(ValueError, match="ws"):
        upipe.qk_norm_rope_bwd(r, q, None, w, None, q, None, q.clone(), None, w.clone(), None,
                               ws=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    with pytest.raises(upipe.UpipeError):
        upipe.qk_norm_rope_fwd(r, q, None, w, None, q, None, eps=-1.0)
    with pytest.raises(upipe.UpipeError):
        upipe.qk_norm_rope_fwd(r, q, None, w, None, q, None, eps=math.nan)
    empty = torch.empty(0, 2, 128, dtype=torch.bfloat16, device="cuda")
    with pytest.raises((upipe.UpipeError, ValueError)):
        upipe.rope_forward(r, empty)


@pytest.mark.parametrize("L,H,Hkv,d,rot,layout", [(1, 1, 1, 128, 128, "half"), (1, 3, 2, 128, 128, "interleaved"),
                                                  (40, 2, 5, 72, 40, "half"), (700, 1, 9, 128, 64, "half"),
                                                  (5000, 2, 2, 64, 64, "interleaved"), (30, 3, 3, 128, 34, "half")])
def test_keys_after_queries_equal_keys_alone(L, H, Hkv, d, rot, layout):
    """The keys take the copies' ring over from the queries: their gradients
    have the bits that they have as the queries of a call of their own."""
    q, k, dq, dk = _randn(21, L, H, d), _randn(22, L, Hkv, d), _randn(23, L, H, d), _randn(24, L, Hkv, d)
    w = torch.linspace(0.5, 1.5, d, device="cuda")
    r = upipe.Rope(d, rot=rot, layout=layout)
    want = upipe.qk_norm_rope_backward(r, k, None, w, None, dk, None, pos0=3)
    x, dy, f = f64(k), f64(dk), np.array(r.freqs)
    _, want_w, size = loc.norm_rope_bwd(x, f64(w), 1e-6, dy, np.arange(L) + 3, f, rot, layout)
    rr = 1 / np.sqrt(np.mean(x * x, -1, keepdims=True) + 1e-6)
    slack = WEIGHT * (size + np.sum(_pair_size(dy, rot, layout) * np.abs(x) * rr, (0, 1)))
    for _ in range(20):
        got = upipe.qk_norm_rope_backward(r, q, k, w, w, dq, dk, pos0=3)
        assert torch.equal(got[1], want[0])
        assert np.all(np.abs(f64(got[3]) - want_w) <= slack)


def _check_norm_backward(q, k, wq, wk, dq, dk, rope, eps, got, name=""):
    """(dq, dk, dwq, dwk) of one call at positions 0, 1, ... against the oracle."""
    pos, f = np.arange(q.shape[0]), np.array(rope.freqs)
    for x, w, dy, dx, dw, n in ((q, wq, dq, got[0], got[2], "q"), (k, wk, dk, got[1], got[3], "k")):
        x, w, dy = f64(x), f64(w), f64(dy)
        want, want_w, size_w = loc.norm_rope_bwd(x, w, eps, dy, pos, f, rope.rot, rope.layout)
        rr = 1 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
        pair = _pair_size(dy, rope.rot, rope.layout)
        dn = np.abs(w) * pair
        _near(dx, want, NORM * rr * (dn + np.abs(x) * rr * np.mean(dn * np.abs(x) * rr, -1, keepdims=True)),
              f"{name} d{n}")
        assert np.all(np.abs(f64(dw) - want_w) <= WEIGHT * (size_w + np.sum(pair * np.abs(x) * rr, (0, 1)))), \
            f"{name} dw{n}"


@pytest.mark.parametrize("d,rot,layout", [(128, 128, "half"), (128, 64, "interleaved"), (64, 64, "half"),
                                          (72, 40, "half"), (24, 8, "interleaved"), (128, 34, "half")])
@pytest.mark.parametrize("H,Hkv", [(1, 2), (6, 3), (5, 7), (16, 1)])
def test_norm_without_eps(d, rot, layout, H, Hkv):
    """eps = 0 with head counts that leave lanes of a step without a head:
    those hold zeros, whose inverse root is infinite, and add nothing."""
    L = 37
    q, k, dq, dk = _randn(25, L, H, d), _randn(26, L, Hkv, d), _randn(27, L, H, d), _randn(28, L, Hkv, d)
    wq, wk = torch.linspace(0.5, 1.5, d, device="cuda"), torch.linspace(1.5, 0.5, d, device="cuda")
    r = upipe.Rope(d, rot=rot, layout=layout)
    f, pos = np.array(r.freqs), np.arange(L)
    for x, w, y in zip((q, k), (wq, wk), upipe.qk_norm_rope_forward(r, q, k, wq, wk, eps=0.0)):
        z = loc.norm_rope(f64(x), f64(w), 0.0, pos, np.zeros(rot // 2), rot, layout)  # unrotated
        _near(y, loc.norm_rope(f64(x), f64(w), 0.0, pos, f, rot, layout), (ANGLE + NORM) * _pair_size(z, rot, layout),
              "forward")
    _check_norm_backward(q, k, wq, wk, dq, dk, r, 0.0, upipe.qk_norm_rope_backward(r, q, k, wq, wk, dq, dk, eps=0.0))


# d, rot, layout: vectors of 8 and of 4 elements in both layouts, single elements; nothing rotated
PARTIAL = [(128, 64, "half"), (128, 34, "interleaved"), (72, 40, "half"), (72, 10, "interleaved"), (128, 34, "half"),
           (16, 2, "half"), (128, 0, "half"), (72, 0, "interleaved"), (256, 48, "half")]


def _bits(t):
    return t.contiguous().view(torch.int16)


@pytest.mark.parametrize("d,rot,layout", PARTIAL)
@pytest.mark.parametrize("transpose", [False, True])
def test_elements_past_rot_are_copied_bit_for_bit(d, rot, layout, transpose):
    """Infinities, NaN of several payloads and zeros of both signs among the
    elements that do not turn stay what they are and reach nothing else."""
    L, H, Hkv = 29, 5, 2
    r = upipe.Rope(d, rot=rot, layout=layout, magnitude=1.25)
    x = [_randn(29, L, H, d), _randn(30, L, Hkv, d)]
    clean = [upipe.rope_forward, upipe.rope_backward][transpose](r, *x, pos0=11)
    g = torch.Generator().manual_seed(31)
    odd = torch.tensor([0x7F80, -0x80, 0x7FC0, 0x7F81, -0x3F, -0x8000, 0, 0x0001], dtype=torch.int16)
    for t in x:
        at = torch.rand(t.shape, generator=g) < 0.3
        at[..., :rot] = False
        _bits(t)[at.cuda()] = odd[torch.randint(0, len(odd), (int(at.sum()),), generator=g)].cuda()
    assert not torch.isfinite(x[0]).all()
    for place in ("apart", "in place"):
        y = [torch.full_like(t, 7.0) for t in x] if place == "apart" else [t.clone() for t in x]
        upipe.rope_apply(r, *(x if place == "apart" else y), *y, pos0=11, transpose=transpose)
        for a, b, c in zip(y, x, clean):
            assert torch.equal(_bits(a)[..., rot:], _bits(b)[..., rot:]), place
            assert torch.equal(_bits(a)[..., :rot], _bits(c)[..., :rot]), place


@pytest.mark.parametrize("d,rot,layout", [p for p in PARTIAL if p[1]])
def test_norm_keeps_elements_past_rot_apart(d, rot, layout):
    """An infinite weight of an element that does not turn makes that element's
    output infinite, and an infinite gradient of it that weight's gradient: no
    other element's, which have the bits that they have without it."""
    L, H, e = 9, 3, d - 3
    r = upipe.Rope(d, rot=rot, layout=layout)
    q, dq, w = _randn(32, L, H, d), _randn(33, L, H, d), torch.linspace(0.5, 1.5, d, device="cuda")
    rest = torch.arange(d, device="cuda") != e
    want, _ = upipe.qk_norm_rope_forward(r, q, None, w, None)
    _, _, want_w, _ = upipe.qk_norm_rope_backward(r, q, None, w, None, dq, None)
    big = w.clone()
    big[e] = math.inf
    y, _ = upipe.qk_norm_rope_forward(r, q, None, big, None)
    assert torch.isinf(y[..., e]).all() and torch.equal(y[..., rest], want[..., rest])
    dq[0, 0, e] = math.inf
    _, _, dw, _ = upipe.qk_norm_rope_backward(r, q, None, w, None, dq, None)
    assert torch.isinf(dw[e]) and torch.equal(dw[rest], want_w[rest])


@pytest.mark.parametrize("d,rot,layout", [(128, 128, "half"), (72, 40, "interleaved"), (128, 34, "half")])
def test_weights_at_any_place_of_a_flat_buffer(d, rot, layout):
    """Weights and their gradients are read and written element by element:
    views into a flat buffer need no alignment but their own."""
    q, k, dq, dk = _randn(34, 50, 3, d), _randn(35, 50, 2, d), _randn(36, 50, 3, d), _randn(37, 50, 2, d)
    flat = torch.linspace(0.5, 1.5, 2 * d + 4, device="cuda")
    wq, wk = flat[1:d + 1], flat[d + 2:2 * d + 2]
    assert wq.data_ptr() % 16 == 4 and wk.data_ptr() % 16 == 8
    r = upipe.Rope(d, rot=rot, layout=layout)
    for a, b in zip(upipe.qk_norm_rope_forward(r, q, k, wq, wk),
                    upipe.qk_norm_rope_forward(r, q, k, wq.clone(), wk.clone())):
        assert torch.equal(a, b)
    want = upipe.qk_norm_rope_backward(r, q, k, wq.clone(), wk.clone(), dq, dk)
    grads = torch.full((2 * d + 4,), 7.0, device="cuda")
    gq, gk = torch.empty_like(q), torch.empty_like(k)
    upipe.qk_norm_rope_bwd(r, q, k, wq, wk, dq, dk, gq, gk, grads[1:d + 1], grads[d + 2:2 * d + 2])
    for a, b in zip((gq, gk, grads[1:d + 1], grads[d + 2:2 * d + 2]), want):
        assert torch.equal(a, b)
    assert (grads[[0, d + 1, 2 * d + 2, 2 * d + 3]] == 7).all()


def test_keys_without_heads():
    """k of no heads is no keys: its weight's gradient, a sum of nothing, is
    written like any other."""
    q, dq, w = _randn(38, 20, 2, 128), _randn(39, 20, 2, 128), torch.ones(128, device="cuda")
    none = q[:, :0]
    r = upipe.Rope(128)
    want = upipe.qk_norm_rope_backward(r, q, None, w, None, dq, None)
    gq, gwq, gwk = torch.empty_like(q), torch.empty_like(w), torch.full_like(w, 7.0)
    upipe.qk_norm_rope_bwd(r, q, none, w, w, dq, none, gq, none, gwq, gwk)
    assert torch.equal(gq, want[0]) and torch.equal(gwq, want[2]) and not gwk.any()
    st = torch.cuda.Stream()
    gwk.fill_(7.0)
    torch.cuda.synchronize()
    upipe.qk_norm_rope_bwd(r, q, none, w, w, dq, none, gq, none, gwq, gwk, stream=st)
    st.synchronize()
    assert not gwk.any()
    y, z = upipe.qk_norm_rope_forward(r, q, none, w, w)
    assert z.shape == none.shape and torch.equal(y, upipe.qk_norm_rope_forward(r, q, None, w, None)[0])


@pytest.mark.parametrize("d,rot,layout", [(128, 128, "interleaved"), (128, 34, "interleaved"), (72, 72, "interleaved"),
                                          (72, 10, "interleaved"), (128, 34, "half"), (24, 18, "half")])
def test_strided_and_in_place_calls_on_the_other_paths(d, rot, layout):
    """The interleaved layouts' vectors of 8 and of 4, and single elements: out
    of and into slices of a fused buffer, head-major outputs, in place."""
    L, H, Hkv = 61, 5, 3
    qkv, dqkv = _fused(40, L, H, Hkv, d), _fused(41, L, H, Hkv, d)
    parts = lambda t: (t[:, :H], t[:, H:H + Hkv])  # noqa: E731
    w = (torch.linspace(0.5, 1.5, d, device="cuda"), torch.linspace(1.5, 0.5, d, device="cuda"))
    r = upipe.Rope(d, rot=rot, layout=layout)
    dense, ddense = ([t.contiguous() for t in parts(x)] for x in (qkv, dqkv))
    runs = [(upipe.rope_forward(r, *dense, pos0=5), lambda x, y: upipe.rope_apply(r, *x, *y, pos0=5)),
            (upipe.rope_backward(r, *dense, pos0=5), lambda x, y: upipe.rope_apply(r, *x, *y, pos0=5, transpose=True)),
            (upipe.qk_norm_rope_forward(r, *dense, *w), lambda x, y: upipe.qk_norm_rope_fwd(r, *x, *w, *y))]
    for want, call in runs:
        buf, hm = qkv.clone(), torch.full((H + Hkv, L, d), 7.0, dtype=torch.bfloat16, device="cuda")
        for src, out in ((qkv, torch.full_like(qkv, 7.0)), (buf, buf)):
            call(parts(src), parts(out))
            assert all(torch.equal(a, b) for a, b in zip(parts(out), want))
        assert torch.equal(buf[:, H + Hkv:], qkv[:, H + Hkv:])
        call(parts(qkv), (hm[:H].transpose(0, 1), hm[H:].transpose(0, 1)))
        assert all(torch.equal(a.transpose(0, 1), b) for a, b in zip((hm[:H], hm[H:]), want))
    want = upipe.qk_norm_rope_backward(r, *dense, *w, *ddense)
    for over in ("gradients", "inputs"):
        x, dy = qkv.clone(), dqkv.clone()
        out, dw = parts(dy if over == "gradients" else x), [torch.empty_like(t) for t in w]
        upipe.qk_norm_rope_bwd(r, *parts(x), *w, *parts(dy), *out, *dw)
        assert all(torch.equal(a, b) for a, b in zip((*out, *dw), want)), over
