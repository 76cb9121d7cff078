"""Pins of the oracle of rotary positions, query/key norms and windowed
attention (oracle/local_oracle.py) against things other than itself: complex
multiplication, torch float64 autograd, finite differences, closed forms and
the full causal oracle; and the host side of the library's rotary tables."""

import math

import numpy as np
import pytest
import torch

from headwise_chunked_context_gb300 import upipe
from oracle import local_oracle as loc
from oracle import upipe_oracle as orc

R = np.random.default_rng


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rot", [(8, 8), (16, 6), (12, 0), (16, 2)])
def test_rope_is_complex_multiplication_and_its_transpose_undoes_it(layout, d, rot):
    x = R(0).standard_normal((5, 3, d))
    pos = np.array([0, 1, 7, -4, 1 << 20])
    f = loc.frequencies(rot) if rot else np.zeros(0)
    y = loc.rope(x, pos, f, rot, layout, magnitude=1.5)
    a, b = loc.pairs(rot, layout)
    z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * pos[:, None, None] * f) * 1.5
    np.testing.assert_allclose(y[..., a], z.real, atol=1e-12)
    np.testing.assert_allclose(y[..., b], z.imag, atol=1e-12)
    assert np.array_equal(y[..., rot:], x[..., rot:])
    back = loc.rope(y, pos, f, rot, layout, magnitude=1.5, transpose=True)
    np.testing.assert_allclose(back[..., :rot], 2.25 * x[..., :rot], atol=1e-12)


def test_frequencies_of_the_scalings():
    f = loc.frequencies(8, theta=16.0)
    np.testing.assert_allclose(f, [1.0, 0.5, 0.25, 0.125])
    np.testing.assert_allclose(loc.frequencies(8, 16.0, ("linear", 4.0)), f / 4)
    # turns in 16 pi positions: 8, 4, 2, 1: above 4 kept, at 1 divided, 2 blended by 1/3
    got = loc.frequencies(8, 16.0, ("bands", 4.0, 1.0, 4.0, 16 * math.pi))
    np.testing.assert_allclose(got, [1.0, 0.5, 0.25 * (1 / 3 + 2 / 3 / 4), 0.125 / 4])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_norm_rope_gradients_match_torch_autograd_and_differences(layout):
    r = R(1)
    L, n, d, rot = 6, 2, 12, 8
    x, w, dy = r.standard_normal((L, n, d)), 1 + 0.1 * r.standard_normal(d), r.standard_normal((L, n, d))
    pos, f = np.arange(L) + 3, loc.frequencies(rot, 100.0)
    dx, dw, mag = loc.norm_rope_bwd(x, w, 1e-3, dy, pos, f, rot, layout, 0.7)
    tx, tw = torch.tensor(x, requires_grad=True), torch.tensor(w, requires_grad=True)
    z = tx * torch.rsqrt(tx.square().mean(-1, keepdim=True) + 1e-3) * tw
    a, b = loc.pairs(rot, layout)
    ang = torch.tensor(pos[:, None] * f)[:, None]
    u = torch.complex(z[..., a], z[..., b]) * torch.polar(torch.full_like(ang, 0.7), ang)
    loss = (u.real * torch.tensor(dy[..., a])).sum() + (u.imag * torch.tensor(dy[..., b])).sum() + \
        (z[..., rot:] * torch.tensor(dy[..., rot:])).sum()
    loss.backward()
    np.testing.assert_allclose(dx, tx.grad.numpy(), atol=1e-12)
    np.testing.assert_allclose(dw, tw.grad.numpy(), atol=1e-12)
    assert np.all(mag >= np.abs(dw) - 1e-12)
    fn = lambda x_, w_: float(np.sum(loc.norm_rope(x_, w_, 1e-3, pos, f, rot, layout, 0.7) * dy))  # noqa: E731
    v, u = r.standard_normal(x.shape), r.standard_normal(d)
    e = 1e-6
    np.testing.assert_allclose((fn(x + e * v, w) - fn(x - e * v, w)) / (2 * e), np.sum(dx * v), rtol=1e-6)
    np.testing.assert_allclose((fn(x, w + e * u) - fn(x, w - e * u)) / (2 * e), np.sum(dw * u), rtol=1e-6)


def test_window_mask_by_hand():
    got = loc.visible(np.arange(5), np.arange(5), window=2, sinks=1).astype(int)
    assert got.tolist() == [[1, 0, 0, 0, 0], [1, 1, 0, 0, 0], [1, 1, 1, 0, 0], [1, 0, 1, 1, 0], [1, 0, 0, 1, 1]]


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 2), (3, 0), (4, 2), (9, 1), (100, 0), (2, 50)])
def test_window_matches_torch_autograd(window, sinks):
    r = R(2)
    L, H, Hkv, d = 17, 4, 2, 8
    q, k, v, do = (r.standard_normal((L, h, d)) for h in (H, Hkv, Hkv, H))
    o, lse = loc.window_fwd(q, k, v, window, sinks)
    dq, dk, dv = loc.window_bwd(q, k, v, o, do, window, sinks)
    t = [torch.tensor(x, requires_grad=True) for x in (q, k, v)]
    i, j = torch.arange(L)[:, None], torch.arange(L)[None]
    keep = (j <= i) & ((j > i - window) | (j < sinks))
    kk, vv = (x.repeat_interleave(H // Hkv, 1).transpose(0, 1) for x in t[1:])
    y = torch.nn.functional.scaled_dot_product_attention(t[0].transpose(0, 1), kk, vv, attn_mask=keep).transpose(0, 1)
    y.backward(torch.tensor(do))
    np.testing.assert_allclose(o, y.detach().numpy(), atol=1e-12)
    for got, x in zip((dq, dk, dv), t):
        np.testing.assert_allclose(got, x.grad.numpy(), atol=1e-12)
    if window >= L or sinks >= L:  # the full causal attention
        fo, fl = orc.attention_core_fwd(q, k, v)
        np.testing.assert_allclose(o, fo, atol=1e-12)
        np.testing.assert_allclose(lse, fl, atol=1e-12)
    if window == 1 and not sinks:  # each query sees itself alone
        np.testing.assert_allclose(o, np.repeat(v, 2, 1), atol=1e-12)


# ------------------------------------------------ the library's host side

@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(upipe.LIB_PATH):
        from headwise_chunked_context_gb300 import build
        build.build()
    return upipe.lib()


@pytest.mark.parametrize("scaling", [None, ("linear", 4.0), ("bands", 8.0, 1.0, 4.0, 8192)])
@pytest.mark.parametrize("rot", [2, 10, 128, 256])
def test_rope_table_holds_the_frequencies(lib, rot, scaling):
    r = upipe.Rope(256, rot=rot, theta=500000.0, scaling=scaling)
    f = loc.frequencies(rot, 500000.0, scaling)
    np.testing.assert_allclose(r.freqs, f, rtol=1e-14)
    # step / 2^64 turns per position, modulo one turn, cut off at 2^-64
    steps = np.array([int(r.table.step[i]) for i in range(rot // 2)], dtype=np.float64) / 2.0 ** 64
    np.testing.assert_allclose(steps, (f / (2 * np.pi)) % 1.0, rtol=1e-14, atol=2.0 ** -64)


def test_rope_table_turns_are_exact_at_far_positions(lib):
    """The wrapping 64-bit product of the table's step and a position is the
    angle: against 80-digit arithmetic, off by no more than the position
    times half a step of the frequency's fp64 value (and of pi's)."""
    from decimal import Decimal, getcontext
    getcontext().prec = 80
    two_pi = Decimal("6.28318530717958647692528676655900576839433879875021164194988918461563281257241799725606965068")
    r = upipe.Rope(128)
    for p in (1, 12345, (1 << 21) + 7, (1 << 31) - 1, -5, -(1 << 31)):
        for i in (0, 1, 17, 63):
            turn = (int(r.table.step[i]) * p) % (1 << 64) / 2.0 ** 64
            want = float((Decimal(r.freqs[i]) * p / two_pi) % 1) % 1.0
            off = abs(turn - want)
            off = min(off, 1 - off)
            assert off <= abs(p) * (r.freqs[i] / (2 * math.pi) * 2.0 ** -52 + 2.0 ** -64) + 2.0 ** -52


def test_rope_given_frequencies_negative_and_large(lib):
    r = upipe.Rope(16, rot=6, freqs=[-0.25, 1e-300, 1000.0])
    got = [int(r.table.step[i]) / 2.0 ** 64 for i in range(3)]
    np.testing.assert_allclose(got, [1 - 0.25 / (2 * math.pi), 0.0, (1000.0 / (2 * math.pi)) % 1.0], rtol=1e-13)
    assert int(upipe.Rope(8, rot=2, freqs=[-1e-300]).table.step[0]) == 0  # 1 - 1e-300 turns is one turn


@pytest.mark.parametrize("kw", [
    dict(d=12), dict(d=0), dict(d=264), dict(d=64, rot=66), dict(d=64, freqs=[math.inf] * 32),
    dict(d=64, magnitude=math.nan), dict(d=64, magnitude=1e31), dict(d=64, theta=0.0), dict(d=64, theta=math.inf),
    dict(d=64, scaling=("linear", 0.0)), dict(d=64, scaling=("bands", 8.0, 4.0, 1.0, 8192)),
    dict(d=64, scaling=("bands", 8.0, 1.0, 4.0, 0)),
])
def test_rope_refuses_what_it_cannot_hold(lib, kw):
    with pytest.raises((upipe.UpipeError, ValueError)):
        upipe.Rope(**kw)


@pytest.mark.parametrize("kw", [
    dict(rot=5), dict(rot=-2), dict(layout="pairs"), dict(scaling=("cubic", 2.0)), dict(scaling=("linear",)),
    dict(freqs=[1.0]), dict(freqs=[1.0] * 64, scaling=("linear", 2.0)),
])
def test_rope_binding_refuses(lib, kw):
    with pytest.raises(ValueError):
        upipe.Rope(128, **kw)


def test_qk_binding_refuses_before_any_launch(lib):
    """CPU tensors: nothing can launch."""
    n0 = upipe.launch_count()
    r = upipe.Rope(128)
    q, k = torch.zeros(4, 8, 128, dtype=torch.bfloat16), torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    w = torch.ones(128)
    for bad in (q.float(), q[:, :, :64], q[0], q.transpose(0, 2), q[:3]):
        with pytest.raises(ValueError):
            upipe.rope_apply(r, q, k, bad, k)
    with pytest.raises(ValueError, match="16-byte"):
        upipe.rope_apply(r, torch.zeros(4, 8, 129, dtype=torch.bfloat16)[:, :, 1:], None, q, None)
    with pytest.raises(ValueError, match="16-byte"):
        upipe.rope_apply(r, torch.zeros(4, 8, 132, dtype=torch.bfloat16)[:, :, :128], None, q, None)
    with pytest.raises(ValueError, match="CUDA"):
        upipe.rope_apply(r, q, k, q, k)
    with pytest.raises(ValueError, match="pos0"):
        upipe.rope_apply(r, q, k, q, k, pos0=3, positions=torch.zeros(4, dtype=torch.int32))
    for bad in (torch.zeros(4, dtype=torch.int64), torch.zeros(3, dtype=torch.int32)):
        with pytest.raises(ValueError, match="positions"):
            upipe.rope_apply(r, q, k, q, k, positions=bad)
    with pytest.raises(ValueError):
        upipe.qk_norm_rope_fwd(r, q, k, w.double(), w, q, k)
    with pytest.raises(ValueError):
        upipe.qk_norm_rope_bwd(r, q, k, w, w, q, k, q, k, w[:64], w)
    assert upipe.launch_count() == n0


def _entry(lib, r, **kw):
    """upipe_rope_apply on made-up aligned addresses; what is wrong is
    refused before the device is asked for."""
    import ctypes
    a = dict(L=4, H=2, Hkv=1, pos0=0, q=(1 << 20, 256, 128), k=(1 << 21, 128, 128), qo=(1 << 22, 256, 128),
             ko=(1 << 23, 128, 128), transpose=0)
    a.update(kw)
    ref = lambda t: ctypes.byref(upipe.Rows(*t)) if t else None  # noqa: E731
    c = upipe.QkCfg(a["L"], a["H"], a["Hkv"], a["pos0"], 0.0)
    return lib.upipe_rope_apply(r._ref, ctypes.byref(c), ref(a["q"]), ref(a["k"]), None, ref(a["qo"]), ref(a["ko"]),
                                a["transpose"], None)


@pytest.mark.skipif(torch.cuda.is_available(), reason="the accepted calls would launch on made-up addresses")
def test_rope_entry_refuses_bad_shapes_pointers_and_strides(lib):
    r = upipe.Rope(128)
    bad = [dict(L=0), dict(L=1 << 31), dict(H=0), dict(H=65537), dict(Hkv=-1), dict(pos0=1 << 62),
           dict(q=None), dict(qo=None), dict(k=None), dict(ko=None), dict(q=(0, 256, 128)), dict(q=((1 << 20) + 8, 256, 128)),
           dict(q=(1 << 20, 260, 128)), dict(q=(1 << 20, -256, 128)), dict(q=(1 << 20, 1 << 62, 128)),
           dict(qo=(1 << 22, 128, 128)), dict(qo=(1 << 22, 256, 64)), dict(qo=(1 << 22, 0, 128)),
           dict(qo=(1 << 22, 128, 256)), dict(transpose=2)]
    for kw in bad:
        assert _entry(lib, r, **kw) == upipe.UPIPE_ERR_INVALID_ARG, kw
    # without a GPU an accepted call ends at the device check
    for kw in (dict(), dict(k=None, ko=None, Hkv=0), dict(qo=(1 << 22, 128, 512)), dict(q=(1 << 20, 0, 0)),
               dict(qo=(1 << 22, 4096, 136))):
        assert _entry(lib, r, **kw) in (upipe.UPIPE_ERR_CUDA, upipe.UPIPE_ERR_UNSUPPORTED_DEVICE), kw
    assert lib.upipe_qk_norm_rope_workspace_bytes(r._ref, None) == 0
    assert upipe.qk_norm_rope_workspace_bytes(r, 1 << 20, 32, 8) == 304 * 2 * 128 * 4
    assert upipe.qk_norm_rope_workspace_bytes(r, 0, 32, 8) == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="the accepted calls would launch on made-up addresses")
def test_norm_entries_take_weights_at_any_float(lib):
    import ctypes
    r, c = upipe.Rope(128), ctypes.byref(upipe.QkCfg(4, 2, 1, 0, 1e-6))
    q, k = ctypes.byref(upipe.Rows(1 << 20, 256, 128)), ctypes.byref(upipe.Rows(1 << 21, 128, 128))
    fwd = lambda wq, wk: lib.upipe_qk_norm_rope_fwd(r._ref, c, q, k, wq, wk, None, q, k, None)  # noqa: E731
    bwd = lambda *w: lib.upipe_qk_norm_rope_bwd(r._ref, c, q, k, w[0], w[1], None, q, k, q, k, w[2], w[3],  # noqa: E731
                                                1 << 24, 1 << 20, None)
    at = 1 << 23
    for entry, n in ((fwd, 2), (bwd, 4)):
        for off in (0, 4, 8, 12):
            assert entry(*[at + off] * n) in (upipe.UPIPE_ERR_CUDA, upipe.UPIPE_ERR_UNSUPPORTED_DEVICE), off
        for i in range(n):
            for bad in (None, at + 2):
                w = [at] * n
                w[i] = bad
                assert entry(*w) == upipe.UPIPE_ERR_INVALID_ARG, (i, bad)


@pytest.mark.parametrize("kw", [dict(window=0), dict(window=-3), dict(sinks=-1), dict(L=0), dict(L=1 << 31), dict(d=64),
                                dict(H=6, Hkv=4), dict(H=96, Hkv=8), dict(Hkv=0)])
def test_window_refuses_bad_configurations(lib, kw):
    import ctypes
    base = dict(L=64, H=4, Hkv=2, window=9, sinks=1)
    cfg = upipe.WindowConfig(**{**base, **kw})
    assert upipe.window_workspace_bytes(cfg) == 0
    a = [ctypes.c_void_p(1 << (20 + i)) for i in range(9)]
    assert lib.upipe_window_fwd(ctypes.byref(cfg.c()), *a[:5], None) == upipe.UPIPE_ERR_INVALID_ARG
    assert lib.upipe_window_bwd(ctypes.byref(cfg.c()), *a, a[0], 1 << 30, None) == upipe.UPIPE_ERR_INVALID_ARG


def test_window_refuses_bad_pointers_and_workspaces(lib):
    import ctypes
    cfg = upipe.WindowConfig(L=200, H=4, Hkv=2, window=9, sinks=1)
    c = ctypes.byref(cfg.c())
    a = [ctypes.c_void_p(1 << (20 + i)) for i in range(9)]
    for i in range(5):
        for bad in (None, ctypes.c_void_p((1 << 20) + 8)):
            b = list(a[:5])
            b[i] = bad
            assert lib.upipe_window_fwd(c, *b, None) == upipe.UPIPE_ERR_INVALID_ARG
    need = upipe.window_workspace_bytes(cfg)
    assert need > 0
    for i in range(9):
        b = list(a)
        b[i] = ctypes.c_void_p((1 << 20) + 4)
        assert lib.upipe_window_bwd(c, *b, a[0], need, None) == upipe.UPIPE_ERR_INVALID_ARG
    assert lib.upipe_window_bwd(c, *a, None, need, None) == upipe.UPIPE_ERR_INVALID_ARG
    assert lib.upipe_window_bwd(c, *a, a[0], need - 1, None) == upipe.UPIPE_ERR_WS_TOO_SMALL


def test_window_binding_refuses_before_any_launch(lib):
    n0 = upipe.launch_count()
    cfg = upipe.WindowConfig(L=64, H=4, Hkv=2, window=9, sinks=1)
    q, k = torch.zeros(64, 4, 128, dtype=torch.bfloat16), torch.zeros(64, 2, 128, dtype=torch.bfloat16)
    lse = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="q"):
        upipe.window_fwd(cfg, q[:63], k, k, q, lse)
    with pytest.raises(ValueError, match="lse"):
        upipe.window_fwd(cfg, q, k, k, q, lse.double())
    with pytest.raises(ValueError, match="dk"):
        upipe.window_bwd(cfg, q, k, k, q, lse, q, q, q, k)
    with pytest.raises(ValueError, match="CUDA"):
        upipe.window_fwd(cfg, q, k, k, q, lse)
    assert upipe.launch_count() == n0


def test_copies_and_pickles_keep_the_tables(lib):
    import copy
    import pickle
    r = upipe.Rope(128, rot=64, layout="interleaved", scaling=("bands", 8.0, 1.0, 4.0, 8192), magnitude=1.25)
    c = upipe.WindowConfig(L=64, H=4, Hkv=2, window=9, sinks=1)
    for f in (copy.deepcopy, copy.copy, lambda x: pickle.loads(pickle.dumps(x))):
        q = f(r)
        assert bytes(q.table) == bytes(r.table) and q.freqs == r.freqs and q.layout == r.layout
        assert f(c) == c and upipe.window_workspace_bytes(f(c)) == upipe.window_workspace_bytes(c)


def test_numbers_past_the_librarys_integers_are_refused(lib):
    q = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    for bad in (1 << 62, -(1 << 62), 1 << 70):
        with pytest.raises(ValueError, match="pos0"):
            upipe.rope_apply(upipe.Rope(128), q, None, q, None, pos0=bad)
    with pytest.raises(ValueError, match="window"):
        upipe.WindowConfig(L=64, H=4, Hkv=2, window=1 << 63)
    with pytest.raises(ValueError, match="sinks"):
        upipe.WindowConfig(L=64, H=4, Hkv=2, window=4, sinks=1 << 64)


def test_window_workspace_shares_of_sinks(lib):
    """32 bytes per query and head, 128 of counters, and fp32 shares of the
    sinks' dK and dV only where later queries are cut into chunks."""
    need = lambda **kw: upipe.window_workspace_bytes(upipe.WindowConfig(**kw))  # noqa: E731
    assert need(L=32768, H=32, Hkv=8, window=4096) == 128 + 32768 * 32 * 32
    # the first tile's 223 later query tiles are less than half of what an SM gets: no cut
    assert need(L=32768, H=32, Hkv=8, window=4096, sinks=4) == 128 + 32768 * 32 * 32
    # 1015 later tiles; (1024 * 9 + 1015) / 304 -> chunks of 34, 30 shares and the tile's own, 16 rows each
    assert need(L=131072, H=8, Hkv=1, window=1024, sinks=16) == 128 + 131072 * 8 * 32 + 31 * 2 * 16 * 128 * 4
    assert need(L=131072, H=8, Hkv=1, window=131072, sinks=16) == 128 + 131072 * 8 * 32


def test_sizes_past_32_bits_are_refused(lib):
    """A C int of (1 << 32) + n is n."""
    for kw in (dict(H=(1 << 32) + 4), dict(Hkv=(1 << 32) + 2), dict(d=(1 << 32) + 128)):
        with pytest.raises(ValueError, match="32 bits"):
            upipe.WindowConfig(**{**dict(L=64, H=4, Hkv=2, window=4), **kw})
    q = torch.zeros(1, 1, 8, dtype=torch.bfloat16)
    for bad in (q.expand(1, (1 << 32) + 1, 8), q.expand(1, 65537, 8)):
        with pytest.raises(ValueError, match="heads"):
            upipe.rope_apply(upipe.Rope(8), bad, None, bad, None)


def test_no_workspace_for_sizes_past_the_librarys_integers(lib):
    r = upipe.Rope(128)
    need = upipe.qk_norm_rope_workspace_bytes
    assert need(r, 100, 8, 2) > 0
    for kw in (dict(L=(1 << 64) + 100), dict(L=1 << 31), dict(H=(1 << 32) + 8), dict(Hkv=(1 << 32) + 2),
               dict(H=8 - (1 << 32))):
        assert need(r, **{**dict(L=100, H=8, Hkv=2), **kw}) == 0, kw


def test_strides_of_axes_of_one_say_nothing(lib):
    """One token of rows of 100 elements, one head of such rows: what would be
    the strides of a second token or head are no multiples of 8."""
    x = torch.zeros(1, 108, dtype=torch.bfloat16)
    for t, L in ((x[:, :72].unsqueeze(1), 1), (torch.zeros(3, 72, dtype=torch.bfloat16).as_strided((3, 1, 72), (72, 100, 1)), 3)):
        assert max(t.stride()) % 8
        rows = upipe._rows(t, L, 1, 72, "q", -1)._obj
        assert rows.p == t.data_ptr() and rows.row % 8 == 0 and rows.head % 8 == 0
    with pytest.raises(ValueError, match="16-byte"):
        upipe._rows(torch.zeros(2, 108, dtype=torch.bfloat16)[:, :72].unsqueeze(1), 2, 1, 72, "q", -1)
