"""GPU parity of token embedding, dropout and layer / RMS norm against the
fp64 oracle, element by element.

Tolerances.  A bf16 output is rounded once, by at most 2^-8 of its size (half
a step).  An fp32 sum of n terms in any order is off by at most n 2^-24 of the
sum of their sizes; the norm's sums over a row of D <= 16384 go through at most
100 additions one after another (64 in a lane, 5 and at most 31 over lanes and
warps): SUM = 1e-5 of the terms' sizes, which covers their own two roundings.
From there on: the mean is off by SUM mean|s|, so n = (s - m) r by r SUM mean|s|,
and by 2 SUM of itself (r: half of its sum's error, and 2 units of 2^-23 of an
inverse root); a product or sum after that adds 2^-23 of its terms' sizes.
A column's sum over L rows of a backward adds, at the tests' sizes, at most 90
terms one after another and 32 shares: SUM of the terms' sizes as well."""

import numpy as np
import pytest
import torch

from headwise_chunked_context_gb300 import upipe
from oracle import residual_oracle as res
from tests.gpu_common import ensure_lib, f64, status_ok

pytestmark = pytest.mark.gpu

HALF_STEP = 2.0 ** -8
SUM = 1e-5
UNIT = 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _randn(seed, *shape, std=1.0, mean=0.0):
    return (torch.randn(*shape, generator=_gen(seed)) * std + mean).to(torch.bfloat16).cuda()


def _near(got, want, slack, name, rounded=True):
    got = f64(got)
    assert np.all(np.isfinite(got)), name
    over = np.abs(got - want) - slack - (HALF_STEP * (np.abs(want) + slack) if rounded else 0)
    assert over.max() <= 0, f"{name}: {over.max():.3e} over at {np.unravel_index(over.argmax(), over.shape)}"


def _inside(t, before=8, after=72, fill=7.0):
    """t's values in rows inside a wider buffer; the buffer, and its part."""
    L, D = t.shape
    buf = torch.full((L, before + D + after), fill, dtype=t.dtype, device="cuda")
    buf[:, before:before + D] = t
    return buf, buf[:, before:before + D]


def _frame_kept(buf, D, before=8, fill=7.0):
    return bool((buf[:, :before] == fill).all() and (buf[:, before + D:] == fill).all())


# ----------------------------------------------------------------- dropout

def _near_sum(got, x, r, mask, name):
    """got = bf16(r + drop(x)): the factor, the product and the sum round by
    2^-24 of the terms each."""
    d = res.add(f64(x), **mask) if mask else f64(x)
    want = d if r is None else f64(r) + d
    slack = 3 * 2.0 ** -24 * (np.abs(d) + (0 if r is None else np.abs(f64(r))))
    _near(got, want, slack, name)


@pytest.mark.parametrize("L,D", [(1, 8), (1, 4096), (7, 1000), (333, 264), (5, 24), (64, 16392), (2, 70000)])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 1 - 2.0 ** -20])
def test_dropout_matches_oracle(L, D, p):
    x, r = _randn(1, L, D), _randn(2, L, D, std=3.0)
    mask = dict(p=p, seed=0x0123456789abcdef, call=(5 << 32) + 9, first=8 * 12345678901)
    d = upipe.Dropout(**mask)
    for given in (None, r):
        y = upipe.dropout_forward(d, x, given)
        _near_sum(y, x, given, mask, f"p {p}")
    # the mask itself, bit for bit
    kept = upipe.dropout_forward(d, torch.ones_like(x)) != 0
    assert np.array_equal(kept.cpu().numpy(), res.keep(L, D, **mask))
    assert torch.equal(upipe.dropout_backward(d, x), upipe.dropout_forward(d, x))
    status_ok()


def test_dropout_of_p_zero_is_the_plain_sum():
    x, r = _randn(3, 50, 520), _randn(4, 50, 520)
    d = upipe.Dropout(0.0)
    assert torch.equal(upipe.dropout_forward(d, x), x)
    assert torch.equal(upipe.dropout_forward(d, x, r), (r.float() + x.float()).bfloat16())


def test_dropped_elements_are_zero_whatever_they_held():
    x, r = _randn(5, 9, 1024), _randn(6, 9, 1024)
    kept = torch.from_numpy(res.keep(9, 1024, 0.5, seed=3)).cuda()
    bad = torch.where(kept, x, torch.tensor(float("nan"), dtype=torch.bfloat16, device="cuda"))
    bad[:, ::2] = torch.where(kept, x, torch.tensor(float("-inf"), dtype=torch.bfloat16, device="cuda"))[:, ::2]
    d = upipe.Dropout(0.5, seed=3)
    assert torch.equal(upipe.dropout_forward(d, bad, r), upipe.dropout_forward(d, x, r))
    assert torch.equal(upipe.dropout_forward(d, bad) == 0, ~kept | (x == 0))
    w = torch.ones(1024, device="cuda")
    for a, b in zip(upipe.layer_norm_forward(bad, w, residual=r, dropout=d),
                    upipe.layer_norm_forward(x, w, residual=r, dropout=d)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("L,D", [(1, 64), (77, 1000), (40, 4096)])
def test_dropout_strided_in_place_and_broadcast(L, D):
    x, r = _randn(7, L, D), _randn(8, L, D)
    d = upipe.Dropout(0.3, seed=11, call=2)
    want = upipe.dropout_forward(d, x, r)
    (bx, sx), (br, sr), (by, sy) = _inside(x), _inside(r, 16, 8), _inside(torch.zeros_like(x), 24, 40)
    upipe.dropout_apply(d, sx, sr, sy)
    assert torch.equal(sy, want) and _frame_kept(by, D, 24)
    upipe.dropout_apply(d, sx, sr, sr)
    assert torch.equal(sr, want) and _frame_kept(br, D, 16)
    upipe.dropout_apply(d, sx, r, sx)
    assert torch.equal(sx, want) and _frame_kept(bx, D)
    y = torch.empty_like(x)
    upipe.dropout_apply(d, x, r[:1].expand(L, D), y)
    assert torch.equal(y, upipe.dropout_forward(d, x, r[:1].repeat(L, 1)))


def test_rows_of_ranks_draw_the_whole_tensors_mask():
    x = _randn(9, 96, 1032)
    want = upipe.dropout_forward(upipe.Dropout(0.2, seed=4, call=6), x)
    for lo, hi in ((0, 31), (31, 32), (32, 96)):
        d = upipe.Dropout(0.2, seed=4, call=6, first=lo * 1032)
        assert torch.equal(upipe.dropout_forward(d, x[lo:hi]), want[lo:hi])


def test_step_on_the_device_is_added_to_the_call():
    x, w = _randn(10, 20, 512), torch.ones(512, device="cuda")
    step = torch.tensor([5], device="cuda")
    a, b = upipe.Dropout(0.4, seed=8, call=100, step=step), upipe.Dropout(0.4, seed=8, call=105)
    assert torch.equal(upipe.dropout_forward(a, x), upipe.dropout_forward(b, x))
    for s, t in zip(upipe.layer_norm_forward(x, w, dropout=a), upipe.layer_norm_forward(x, w, dropout=b)):
        assert torch.equal(s, t)
    step -= 6  # wraps past 64 bits: call 99
    assert torch.equal(upipe.dropout_forward(a, x), upipe.dropout_forward(upipe.Dropout(0.4, seed=8, call=99), x))


# -------------------------------------------------------------------- norm

# L, D: one vector a row, rows of less than a warp, of one and many vectors per lane, the largest; one row and
# more rows than are resident
SHAPES = [(1, 8), (1, 5120), (3, 72), (300, 256), (65, 1000), (33, 1032), (129, 4096), (50, 5120), (1, 16384),
          (37, 8192), (19, 16384), (21, 12296), (2501, 128), (1300, 520),
          (1300, 1024), (700, 5120), (701, 2560), (1301, 4096), (399, 7000)]  # several rows a team


def _weights(seed, D):
    g = _gen(seed)
    return (1 + 0.3 * torch.randn(D, generator=g)).cuda(), (0.5 * torch.randn(D, generator=g)).cuda()


def _check_norm(y, s, w, b, eps, rms, name):
    s = f64(s)
    m, r = res.stats(s, eps, rms)
    n = (s - m) * r
    e_n = SUM * ((0 if rms else r * np.abs(s).mean(-1, keepdims=True)) + 2 * np.abs(n))
    w = f64(w)
    want = n * w + (0 if b is None else f64(b))
    _near(y, want, np.abs(w) * e_n + 2 * UNIT * (np.abs(n * w) + np.abs(want)), name)


@pytest.mark.parametrize("L,D", SHAPES)
@pytest.mark.parametrize("rms,bias", [(False, True), (False, False), (True, False), (True, True)])
def test_norm_matches_oracle(L, D, rms, bias):
    x, (w, b) = _randn(L + D, L, D, std=2.0, mean=0.5), _weights(D, D)
    b = b if bias else None
    y, s = upipe.layer_norm_forward(x, w, b, eps=1e-5, rms=rms)
    assert s is x
    _check_norm(y, x, w, b, 1e-5, rms, "y")
    status_ok()


@pytest.mark.parametrize("L,D", SHAPES)
@pytest.mark.parametrize("given,p", [(True, None), (True, 0.0), (True, 0.2), (False, 0.2)])
def test_sum_and_norm_match_oracle(L, D, given, p):
    x, r, (w, b) = _randn(1, L, D), _randn(2, L, D, std=3.0) if given else None, _weights(D, D)
    mask = dict(p=p, seed=77, call=L, first=16) if p is not None else {}
    d = upipe.Dropout(**mask) if mask else None
    y, s = upipe.layer_norm_forward(x, w, b, residual=r, dropout=d)
    _near_sum(s, x, r, mask, "s")
    _check_norm(y, s, w, b, 1e-5, False, "y")
    # one pass gives the bits of two
    if d is not None:
        assert torch.equal(s, upipe.dropout_forward(d, x, r))
    assert torch.equal(y, upipe.layer_norm_forward(s, w, b)[0])
    status_ok()


def _check_norm_bwd(got, s, w, dy, ds, eps, rms, mask):
    dx, dres, dw, db = got
    s, w, dy, ds = f64(s), f64(w), f64(dy), None if ds is None else f64(ds)
    want, want_w, want_b = res.norm_bwd(s, w, dy, ds, eps, rms)
    mean = lambda a: a.mean(-1, keepdims=True)  # noqa: E731
    m, r = res.stats(s, eps, rms)
    n, g = (s - m) * r, dy * w
    e_n = SUM * ((0 if rms else r * mean(np.abs(s))) + 2 * np.abs(n))
    mg, k = (0 if rms else mean(g)), mean(g * n)
    e_mg = 0 if rms else SUM * mean(np.abs(g))
    e_k = 2 * SUM * mean(np.abs(g * n)) + mean(np.abs(g) * e_n)
    size = r * (np.abs(g) + np.abs(mg) + np.abs(n * k))
    slack = r * (e_mg + np.abs(n) * e_k + np.abs(k) * e_n) + 2 * SUM * size + UNIT * (
        size + np.abs(want) + (0 if ds is None else np.abs(ds)))
    _near(dres, want, slack, "dres")
    if mask:
        f = res.drop(np.ones_like(want), **mask)
        _near(dx, want * f, slack * f + 2 * UNIT * np.abs(want * f), "dx")
        assert np.array_equal(f64(dx) == 0, (f == 0) | (f64(dx) == 0)) and not f64(dx)[f == 0].any()
    else:
        assert dx is dres
    _near(dw, want_w, SUM * np.abs(dy * n).sum(0) + (np.abs(dy) * e_n).sum(0), "dw", rounded=False)
    if db is not None:
        _near(db, want_b, SUM * np.abs(dy).sum(0), "db", rounded=False)


@pytest.mark.parametrize("L,D", SHAPES)
@pytest.mark.parametrize("rms,bias,given,p", [(False, True, False, None), (True, False, True, 0.1),
                                              (False, True, True, None), (True, True, False, 0.5),
                                              (False, False, True, 0.0), (False, True, True, 0.3)])
def test_norm_backward_matches_oracle(L, D, rms, bias, given, p):
    s, dy, (w, _) = _randn(3, L, D, std=2.0, mean=-0.5), _randn(4, L, D), _weights(D + 1, D)
    ds = _randn(5, L, D) if given else None
    mask = dict(p=p, seed=78, call=L, first=8) if p is not None else {}
    d = upipe.Dropout(**mask) if mask else None
    got = upipe.layer_norm_backward(s, w, dy, ds, eps=1e-5, rms=rms, bias=bias, dropout=d)
    _check_norm_bwd(got, s, w, dy, ds, 1e-5, rms, mask)
    assert (got[3] is not None) == bias
    if p == 0.0:
        assert torch.equal(got[0], got[1])
    status_ok()


@pytest.mark.parametrize("D", [256, 4096, 1000])
@pytest.mark.parametrize("kind", ["offset", "outlier", "large", "small", "constant", "zero"])
def test_norm_of_rows_that_strain_it(D, kind):
    """A mean far above the spread (the squares' own sum would lose it), single
    channels far above the rest, sizes near the limits of the sums, rows without
    spread."""
    L = 40
    x = _randn(6, L, D)
    if kind == "offset":
        x = x + 100
    if kind == "outlier":
        x[:, 3] *= 1000
        x[::2, D // 2] = -3000
    if kind == "large":
        x = x * 1e14
    if kind == "small":
        x = x * 1e-12
    if kind == "constant":
        x = x[:, :1].expand(L, D).contiguous()
    if kind == "zero":
        x = torch.zeros_like(x)
    (w, b), dy = _weights(7, D), _randn(8, L, D)
    for rms in (False, True):
        y, _ = upipe.layer_norm_forward(x, w, b, rms=rms)
        _check_norm(y, x, w, b, 1e-5, rms, kind)
        _check_norm_bwd(upipe.layer_norm_backward(x, w, dy, rms=rms), x, w, dy, None, 1e-5, rms, {})


def test_rows_with_infinities_and_nan_spoil_no_other_row():
    L, D = 50, 1032
    x, dy, (w, b) = _randn(9, L, D), _randn(10, L, D), _weights(9, D)
    bad = x.clone()
    bad[3, 7], bad[11, 1000], bad[12] = float("inf"), float("nan"), float("-inf")
    good = [i for i in range(L) if i not in (3, 11, 12)]
    y, _ = upipe.layer_norm_forward(bad, w, b)
    assert torch.equal(y[good], upipe.layer_norm_forward(x, w, b)[0][good])
    assert not torch.isfinite(y[[11, 12]].float()).any()
    dx = upipe.layer_norm_backward(bad, w, dy)[0]
    assert torch.equal(dx[good], upipe.layer_norm_backward(x, w, dy)[0][good])


@pytest.mark.parametrize("L,D", [(1, 64), (70, 1000), (40, 4096), (30, 12296)])
@pytest.mark.parametrize("p", [None, 0.3])
def test_norm_strided_in_place_and_off_boundary_weights(L, D, p):
    x, r, dy, ds = (_randn(20 + i, L, D) for i in range(4))
    d = None if p is None else upipe.Dropout(p, seed=12, call=3)
    w, b = _weights(21, D)
    y, s = upipe.layer_norm_forward(x, w, b, residual=r, dropout=d)
    flat = torch.empty(4 * D + 5, device="cuda")  # parameters and gradients inside a flat buffer
    ow, ob, odw, odb = flat[1:1 + D], flat[1 + D:1 + 2 * D], flat[3 + 2 * D:3 + 3 * D], flat[5 + 3 * D:]
    ow.copy_(w)
    ob.copy_(b)
    (bx, sx), (br, sr), (by, sy) = _inside(x), _inside(r, 16, 8), _inside(torch.zeros_like(x), 24, 40)
    upipe.layer_norm_fwd(sx, ow, ob, sy, sr, residual=sr, dropout=d)  # the sum over the residual
    assert torch.equal(sy, y) and torch.equal(sr, s) and _frame_kept(by, D, 24) and _frame_kept(br, D, 16)
    upipe.layer_norm_fwd(x2 := x.clone(), ow, ob, r2 := r.clone(), x2, residual=r2, dropout=d)
    assert torch.equal(r2, y) and torch.equal(x2, s)  # the sum over x, the norm over the residual
    upipe.layer_norm_fwd(x3 := x.clone(), w, b, x3)
    assert torch.equal(x3, upipe.layer_norm_forward(x, w, b)[0])
    want = upipe.layer_norm_backward(s, w, dy, ds, dropout=d)
    (bs, ss), (bd, sd), (be, se) = _inside(s), _inside(dy, 16, 8), _inside(ds, 24, 40)
    upipe.layer_norm_bwd(ss, ow, sd, se, sd, None if d is None else se, odw, odb, dropout=d)
    assert torch.equal(sd, want[1]) and _frame_kept(bd, D, 16) and _frame_kept(be, D, 24) and _frame_kept(bs, D)
    if d is not None:
        assert torch.equal(se, want[0])
    assert torch.equal(odw, want[2]) and torch.equal(odb, want[3]) and torch.equal(ow, w)
    one = ds[:1].expand(L, D)  # one row of gradients for all
    got = upipe.layer_norm_backward(s, w, dy, one)
    for a, c in zip(got, upipe.layer_norm_backward(s, w, dy, ds[:1].repeat(L, 1))):
        assert torch.equal(a, c)


def test_norm_gives_the_same_bits_again_and_by_any_split_of_rows():
    L, D = 3000, 1000
    s, dy, (w, b) = _randn(30, L, D), _randn(31, L, D), _weights(32, D)
    first = upipe.layer_norm_backward(s, w, dy)
    for x, y in zip(first, upipe.layer_norm_backward(s, w, dy)):
        assert torch.equal(x, y)
    y, _ = upipe.layer_norm_forward(s, w, b)
    for lo, hi in ((0, 1), (1, 40), (40, 3000)):  # a row's result does not depend on the others
        assert torch.equal(upipe.layer_norm_forward(s[lo:hi], w, b)[0], y[lo:hi])
        assert torch.equal(upipe.layer_norm_backward(s[lo:hi], w, dy[lo:hi])[0], first[0][lo:hi])


# --------------------------------------------------------------- embedding

def _tokens(seed, L, V, wide, kind="many"):
    g = _gen(seed)
    if kind == "one":
        t = torch.full((L,), V // 2)
    elif kind == "few":
        t = torch.randint(0, min(V, 5), (L,), generator=g)
    else:
        t = torch.randint(0, V, (L,), generator=g)
    return t.to(torch.int64 if wide else torch.int32).cuda()


def _edge(t, V):
    """Padding and tokens past the table among them."""
    t = t.clone()
    if len(t) > 8:
        t[3], t[len(t) // 2], t[-2:] = -1, V, -5
        t[5] = torch.iinfo(t.dtype).max
        t[6] = torch.iinfo(t.dtype).min
    return t


@pytest.mark.parametrize("L,V,D", [(1, 1, 8), (1, 5000, 4096), (300, 512, 256), (77, 1000, 1032), (2000, 37, 72),
                                   (9, 3, 16392)])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_embedding_matches_oracle(L, V, D, wide, dtype):
    W = torch.randn(V, D, generator=_gen(40)).to(dtype).cuda()
    t = _edge(_tokens(41, L, V, wide), V)
    for scale in (1.0, -11.3):
        y = upipe.embed_forward(t, W, scale)
        scale = float(np.float32(scale))
        want = res.embed(t.cpu().numpy(), f64(W), scale)
        assert np.array_equal(np.isnan(f64(y)), np.isnan(want))
        _near(torch.nan_to_num(y), np.nan_to_num(want), 2.0 ** -24 * np.abs(np.nan_to_num(want)), "y")
    if dtype == torch.bfloat16:  # rows as they are
        real = ((t >= 0) & (t < V)).cpu()
        assert torch.equal(upipe.embed_forward(t, W)[real.cuda()], W[t[real.cuda()].long()])
    buf, y = _inside(torch.zeros(L, D, dtype=torch.bfloat16, device="cuda"))
    upipe.embed_fwd(t, W, y, 2.0)
    assert torch.equal(torch.nan_to_num(y), torch.nan_to_num(upipe.embed_forward(t, W, 2.0))) and _frame_kept(buf, D)
    status_ok()


# L, V: one token, fewer tokens than rows and more, tiles of the sort that end inside a part, keys of one to three
# passes (9 bits each), rows with all of the tokens
GRADS = [(1, 1, 8, "many"), (1, 5000, 264, "many"), (2, 511, 64, "many"), (300, 512, 256, "many"),
         (77, 1000, 1032, "many"), (2049, 37, 72, "many"), (5000, 300000, 16, "many"), (6000, 262144, 8, "many"),
         (1025, 40, 1000, "one"), (4099, 3001, 128, "few"), (33, 33, 4096, "one"), (4097, 700, 520, "many"),
         (20000, 9, 24, "many"), (700, 5, 8192, "few"), (40000, 513, 8, "many"), (17000, 20000, 8, "many"),
         # more rows than tokens: zeros beside the sort at the table's end, of all of it and of a part, beside one
         # launch, four and six; the longest rows
         (40, 33000, 1024, "many"), (8192, 8193, 16, "many"), (8200, 17000, 1024, "many"), (8193, 270000, 96, "many"),
         (9000, 9001, 264, "few"), (20, 40, 65536, "many"), (40, 20, 40000, "many")]


@pytest.mark.parametrize("L,V,D,kind", GRADS)
@pytest.mark.parametrize("wide", [False, True])
def test_embedding_gradient_matches_oracle(L, V, D, kind, wide):
    t, dy = _edge(_tokens(42, L, V, wide, kind), V), _randn(43, L, D)
    scale = float(np.float32(1.7))
    want, size, count = res.embed_bwd(t.cpu().numpy(), f64(dy), V, scale)
    # any order of count terms, and the scale's product
    slack = (count[:, None] + 2) * 2.0 ** -24 * size
    got = upipe.embed_backward(t, dy, V, scale)
    _near(got, want, slack, "dW", rounded=False)
    assert not f64(got)[count == 0].any()
    assert torch.equal(got, upipe.embed_backward(t, dy, V, scale))
    # added: rows without a token stay as they are, bit for bit
    base = torch.randn(V, D, generator=_gen(44)).cuda()
    dW = base.clone()
    upipe.embed_bwd(t, dy, dW, scale, add=True)
    none = torch.from_numpy(count == 0).cuda()
    assert torch.equal(dW[none], base[none])
    _near(dW, f64(base) + want, slack + 2.0 ** -24 * (np.abs(f64(base)) + np.abs(want)), "added", rounded=False)
    # rows inside a wider buffer, and one row for all tokens
    _, part = _inside(dy)
    dW = torch.full((V, D), 3.0, device="cuda")
    upipe.embed_bwd(t, part, dW, scale)
    assert torch.equal(dW, got)
    upipe.embed_bwd(t, dy[:1].expand(L, D), dW, scale)
    assert torch.equal(dW, upipe.embed_backward(t, dy[:1].repeat(L, 1), V, scale))
    status_ok()


def test_embedding_gradient_ignores_what_padding_holds():
    t = _tokens(45, 500, 60, False)
    t[::7] = -1
    t[::11] = 60
    dy = _randn(46, 500, 264)
    want = upipe.embed_backward(t, dy, 60)
    dy[::7], dy[::11] = float("nan"), float("inf")
    assert torch.equal(upipe.embed_backward(t, dy, 60), want)
    t[:] = -1  # nothing but padding
    assert not upipe.embed_backward(t, dy, 60).any()


def test_embedding_gradient_writes_nothing_past_its_table():
    t, dy, V, D = _tokens(47, 900, 50, True), _randn(48, 900, 256), 50, 256
    whole = torch.full((V + 2, D), 9.0, device="cuda")
    upipe.embed_bwd(t, dy, whole[1:1 + V], 1.0)
    assert (whole[0] == 9).all() and (whole[-1] == 9).all()
    assert torch.equal(whole[1:1 + V], upipe.embed_backward(t, dy, V))


def test_calls_on_a_stream_of_their_own():
    """The call's stream is the one given, its workspace that stream's."""
    side = torch.cuda.Stream()
    t, dy, w = _tokens(49, 700, 90, False), _randn(50, 700, 520), torch.ones(520, device="cuda")
    want = (upipe.embed_backward(t, dy, 90), *upipe.layer_norm_backward(dy, w, dy, bias=False)[1:3])
    dW, dres, dw, y = torch.zeros_like(want[0]), torch.zeros_like(dy), torch.zeros_like(w), torch.zeros_like(dy)
    torch.cuda.synchronize()
    upipe.embed_bwd(t, dy, dW, stream=side)
    upipe.layer_norm_bwd(dy, w, dy, None, dres, None, dw, None, stream=side)
    upipe.dropout_apply(upipe.Dropout(0.5), dy, None, y, stream=side)
    side.synchronize()
    assert torch.equal(dW, want[0]) and torch.equal(dres, want[1]) and torch.equal(dw, want[2])
    assert torch.equal(y, upipe.dropout_forward(upipe.Dropout(0.5), dy))
    ws = torch.empty(upipe.embed_workspace_bytes(700, 90, 520), dtype=torch.uint8, device="cuda")
    upipe.embed_bwd(t, dy, dW, ws=ws)
    assert torch.equal(dW, want[0])
    with pytest.raises(ValueError, match="ws"):
        upipe.embed_bwd(t, dy, dW, ws=ws[:-16])
    status_ok()


def test_binding_refuses_what_the_kernels_cannot_read():
    x, w, t = _randn(51, 6, 264), torch.ones(264, device="cuda"), _tokens(52, 6, 9, False)
    W, d = torch.zeros(9, 264, device="cuda"), upipe.Dropout(0.1)
    off = torch.empty(6 * 264 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(6, 264)
    n0 = upipe.launch_count()
    for f in (lambda: upipe.dropout_forward(d, off), lambda: upipe.dropout_forward(d, x.t()),
              lambda: upipe.dropout_forward(d, x.float()), lambda: upipe.dropout_forward(d, x, x[:3]),
              lambda: upipe.dropout_apply(d, x, None, x.cpu()), lambda: upipe.dropout_apply(d, x[:, ::2], None, x),
              lambda: upipe.layer_norm_forward(x, w[:8]), lambda: upipe.layer_norm_forward(x, w.double()),
              lambda: upipe.layer_norm_forward(x, torch.ones(528, device="cuda")[::2]),
              lambda: upipe.layer_norm_forward(x, w, residual=off), lambda: upipe.layer_norm_forward(x, w, w.bfloat16()),
              lambda: upipe.layer_norm_backward(x, w, x, off), lambda: upipe.layer_norm_bwd(x, w, x, None, x, x, w, None),
              lambda: upipe.layer_norm_bwd(x, w, x, None, x, None, w, None, dropout=d),
              lambda: upipe.embed_forward(t[::2], W), lambda: upipe.embed_forward(t.cpu(), W),
              lambda: upipe.embed_forward(t, W.t()), lambda: upipe.embed_fwd(t, W, x[:, :256]),
              lambda: upipe.embed_bwd(t, x[:5], W), lambda: upipe.embed_bwd(t, x, W.bfloat16()),
              lambda: upipe.embed_bwd(t, x, W.expand(9, 264)[:, :256])):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: upipe.dropout_forward(d, x[:, :260].contiguous()), lambda: upipe.dropout_forward(d, x[:0]),
              lambda: upipe.layer_norm_forward(x[:0], w), lambda: upipe.layer_norm_forward(x, w, eps=-1.0),
              lambda: upipe.embed_forward(t[:0], W), lambda: upipe.embed_forward(t, W, float("nan")),
              lambda: upipe.dropout_apply(d, x, None, x[:1].expand(6, 264)), lambda: upipe.embed_backward(t, x, 0)):
        with pytest.raises((upipe.UpipeError, ValueError)):
            f()
    assert upipe.launch_count() == n0
