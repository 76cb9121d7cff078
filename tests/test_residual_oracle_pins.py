"""Pins of the residual stream's oracle (CPU): published vectors of the
generator, closed forms and differences of the norm, counting of the
embedding's gradient; and the host's refusals, which reach no device."""

import copy
import ctypes
import os
import pickle

import numpy as np
import pytest
import torch

from headwise_chunked_context_gb300 import upipe
from oracle import residual_oracle as res


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(upipe.LIB_PATH):
        from headwise_chunked_context_gb300 import build
        build.build()
    return upipe.lib()


@pytest.mark.parametrize("counter,key,words", [
    ((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
    ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
    ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
     (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1)),
])
def test_generator_gives_its_authors_vectors(counter, key, words):
    """The known answers that the generator's authors publish with it."""
    assert tuple(int(w) for w in res.philox(counter, key)) == words


def test_mask_counts_elements_from_first_and_by_call():
    whole = res.keep(12, 24, 0.4, seed=99, call=7)
    for r in (0, 1, 5, 11):
        assert np.array_equal(whole[r:], res.keep(12 - r, 24, 0.4, seed=99, call=7, first=24 * r))
    assert not np.array_equal(whole, res.keep(12, 24, 0.4, seed=99, call=8))
    assert not np.array_equal(whole, res.keep(12, 24, 0.4, seed=100, call=7))
    assert res.keep(3, 8, 0.0).all()
    # nested: what p keeps, a smaller p keeps too
    assert not (whole & ~res.keep(12, 24, 0.2, seed=99, call=7)).any()


@pytest.mark.parametrize("p", [0.1, 0.5, 0.9])
def test_mask_keeps_its_share(p):
    """256 x 4096 draws: five standard deviations of a mean."""
    n = 1 << 20
    assert abs(res.keep(256, 4096, p, seed=5, call=3).mean() - (1 - p)) < 5 * np.sqrt(p * (1 - p) / n)


@pytest.mark.parametrize("rms", [False, True])
def test_norm_gradients_by_differences(rms):
    """Central differences of sum(y dy) with a step of 1e-5: off by the third
    derivative's 1e-10 and by 1e-16 / 1e-5 rounding, both scaled by |dy| sqrt(D)."""
    rng = np.random.default_rng(0)
    s, w, b, dy = rng.normal(size=(3, 24)), rng.normal(size=24), rng.normal(size=24), rng.normal(size=(3, 24))
    d, dw, db = res.norm_bwd(s, w, dy, None, 1e-3, rms)
    f = lambda s, w, b: float((res.norm(s, w, b, 1e-3, rms) * dy).sum())  # noqa: E731
    h = 1e-5
    for i in range(3):
        for j in range(0, 24, 5):
            e = np.zeros((3, 24))
            e[i, j] = h
            assert abs((f(s + e, w, b) - f(s - e, w, b)) / (2 * h) - d[i, j]) < 1e-8
    for j in range(24):
        e = np.zeros(24)
        e[j] = h
        assert abs((f(s, w + e, b) - f(s, w - e, b)) / (2 * h) - dw[j]) < 1e-8
        assert abs((f(s, w, b + e) - f(s, w, b - e)) / (2 * h) - db[j]) < 1e-8
    # what reaches s behind the norm adds on
    ds = rng.normal(size=(3, 24))
    assert np.allclose(res.norm_bwd(s, w, dy, ds, 1e-3, rms)[0], d + ds, rtol=0, atol=1e-15)


def test_norm_closed_forms():
    s = np.array([[1.0, -1.0, 1.0, -1.0, 3.0, 3.0, 3.0, 3.0]])
    y = res.norm(s, np.ones(8), None, 0.0, False)
    assert np.allclose(y, (s - 1.5) / np.sqrt(np.var(s)), atol=1e-15)
    assert np.allclose(res.norm(s, np.ones(8), None, 0.0, True), s / np.sqrt(5.0), atol=1e-15)
    # a constant row: the bias
    assert np.array_equal(res.norm(np.full((1, 8), 7.0), np.ones(8), np.arange(8.0), 1e-5, False)[0], np.arange(8.0))


def test_embedding_by_counting():
    W = np.arange(12.0).reshape(4, 3)
    t = np.array([2, -1, 0, 2, 4, -7])
    y = res.embed(t, W, 2.0)
    assert np.array_equal(y[[0, 2, 3]], 2 * W[[2, 0, 2]]) and not y[[1, 5]].any() and np.isnan(y[4]).all()
    dW, size, n = res.embed_bwd(t, np.ones((6, 3)), 4, 2.0)
    assert np.array_equal(dW, np.outer([2, 0, 4, 0], np.ones(3))) and list(n) == [1, 0, 2, 0]
    assert np.array_equal(dW, size)


# --------------------------------------------------------------- refusals

def _rows(p=1 << 20, row=256):
    return ctypes.byref(upipe.Rows(p, row, 0))


GOOD_P = ctypes.c_void_p(1 << 20)  # never dereferenced: rejected first


@pytest.mark.parametrize("bad", [dict(L=0), dict(L=-3), dict(L=1 << 31), dict(V=0), dict(V=-1), dict(D=0), dict(D=12),
                                 dict(D=4), dict(D=65544), dict(wide=2), dict(master=-1), dict(scale=float("nan")),
                                 dict(scale=float("inf"))])
def test_embedding_refuses_bad_sizes(lib, bad):
    c = upipe.EmbedCfg(*({**dict(L=64, V=100, D=256, wide=0, master=1, scale=1.0), **bad}.values()))
    n0 = upipe.launch_count()
    assert lib.upipe_embed_workspace_bytes(ctypes.byref(c)) == 0
    assert lib.upipe_embed_fwd(ctypes.byref(c), GOOD_P, GOOD_P, _rows(), None) == -1
    assert lib.upipe_embed_bwd(ctypes.byref(c), GOOD_P, _rows(), GOOD_P, 0, GOOD_P, 1 << 40, None) == -1
    assert upipe.launch_count() == n0


def test_embedding_refuses_bad_pointers_and_workspaces(lib):
    c = upipe.EmbedCfg(64, 100, 256, 1, 1, 1.0)
    r = ctypes.byref(c)
    n0 = upipe.launch_count()
    odd = ctypes.c_void_p((1 << 20) + 4)  # a 64-bit token's boundary is 8 bytes
    need = lib.upipe_embed_workspace_bytes(r)
    assert need > 0
    for args in ((None, GOOD_P, _rows()), (odd, GOOD_P, _rows()), (GOOD_P, None, _rows()), (GOOD_P, odd, _rows()),
                 (GOOD_P, GOOD_P, None), (GOOD_P, GOOD_P, _rows(row=255)), (GOOD_P, GOOD_P, _rows(row=248)),
                 (GOOD_P, GOOD_P, _rows(p=(1 << 20) + 8)), (GOOD_P, GOOD_P, _rows(row=-256)),
                 (GOOD_P, GOOD_P, _rows(row=1 << 60))):
        assert lib.upipe_embed_fwd(r, *args, None) == -1
    for args in ((None, _rows(), GOOD_P, 0, GOOD_P, need), (GOOD_P, None, GOOD_P, 0, GOOD_P, need),
                 (GOOD_P, _rows(), None, 0, GOOD_P, need), (GOOD_P, _rows(), odd, 0, GOOD_P, need),
                 (GOOD_P, _rows(), GOOD_P, 2, GOOD_P, need), (GOOD_P, _rows(), GOOD_P, 0, None, need)):
        assert lib.upipe_embed_bwd(r, *args, None) == -1
    assert lib.upipe_embed_bwd(r, GOOD_P, _rows(), GOOD_P, 0, GOOD_P, need - 1, None) == upipe.UPIPE_ERR_WS_TOO_SMALL
    assert upipe.launch_count() == n0


@pytest.mark.parametrize("bad", [dict(p=-0.1), dict(p=1.0), dict(p=1 - 2.0 ** -34), dict(p=float("nan")),
                                 dict(first=4), dict(first=1 << 63), dict(step=(1 << 20) + 4)])
def test_masks_out_of_range_are_refused(lib, bad):
    d = upipe.DropoutCfg(*({**dict(p=0.1, seed=1, call=2, first=8, step=None), **bad}.values()))
    n = upipe.NormCfg(4, 256, 0, 1e-5)
    n0 = upipe.launch_count()
    assert lib.upipe_dropout_apply(ctypes.byref(d), 4, 256, _rows(), None, _rows(), None) == -1
    assert lib.upipe_layer_norm_fwd(ctypes.byref(n), ctypes.byref(d), _rows(), None, GOOD_P, None, _rows(), _rows(),
                                    None) == -1
    assert lib.upipe_layer_norm_bwd(ctypes.byref(n), ctypes.byref(d), _rows(), GOOD_P, _rows(), None, _rows(), _rows(),
                                    GOOD_P, None, GOOD_P, 1 << 40, None) == -1
    assert upipe.launch_count() == n0


def test_dropout_refuses_bad_tensors(lib):
    d = ctypes.byref(upipe.DropoutCfg(0.1, 1, 2, 0, None))
    n0 = upipe.launch_count()
    for L, D in ((0, 256), (1 << 31, 256), (4, 0), (4, 252), (4, -8)):
        assert lib.upipe_dropout_apply(d, L, D, _rows(), None, _rows(), None) == -1
    assert lib.upipe_dropout_apply(None, 4, 256, _rows(), None, _rows(), None) == -1
    for x, r, y in ((None, None, _rows()), (_rows(), None, None), (_rows(row=100), None, _rows()),
                    (_rows(), _rows(p=(1 << 20) + 2), _rows()), (_rows(), None, _rows(row=0)),
                    (_rows(), None, _rows(row=248))):
        assert lib.upipe_dropout_apply(d, 4, 256, x, r, y, None) == -1
    assert upipe.launch_count() == n0


@pytest.mark.parametrize("bad", [dict(L=0), dict(L=1 << 31), dict(D=0), dict(D=20), dict(D=16392), dict(rms=2),
                                 dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf"))])
def test_norm_refuses_bad_sizes(lib, bad):
    c = ctypes.byref(upipe.NormCfg(*({**dict(L=4, D=256, rms=0, eps=1e-5), **bad}.values())))
    n0 = upipe.launch_count()
    assert lib.upipe_layer_norm_workspace_bytes(c) == 0
    assert lib.upipe_layer_norm_fwd(c, None, _rows(row=16384), None, GOOD_P, None, None, _rows(row=16384), None) == -1
    assert lib.upipe_layer_norm_bwd(c, None, _rows(row=16384), GOOD_P, _rows(row=16384), None, _rows(row=16384), None,
                                    GOOD_P, None, GOOD_P, 1 << 40, None) == -1
    assert upipe.launch_count() == n0


def test_norm_refuses_bad_pointers_and_sums_that_do_not_fit(lib):
    c = ctypes.byref(upipe.NormCfg(4, 256, 0, 1e-5))
    d = ctypes.byref(upipe.DropoutCfg(0.1, 1, 2, 0, None))
    g, odd, T = GOOD_P, ctypes.c_void_p((1 << 20) + 2), _rows()
    n0 = upipe.launch_count()
    # (drop, x, res, w, b, s, y); s iff a sum
    for a in ((None, None, None, g, None, None, T), (None, T, None, None, None, None, T),
              (None, T, None, odd, None, None, T), (None, T, None, g, odd, None, T), (None, T, None, g, None, None, None),
              (None, T, None, g, None, T, T), (None, T, T, g, None, None, T), (d, T, None, g, None, None, T),
              (None, T, _rows(row=4), g, None, T, T), (None, T, T, g, None, _rows(row=8), T)):
        assert lib.upipe_layer_norm_fwd(c, *a, None) == -1
    need = lib.upipe_layer_norm_workspace_bytes(c)
    # (drop, s, w, dy, ds, dres, dx, dw, db, ws, bytes)
    for a in ((None, None, g, T, None, T, None, g, None, g, need), (None, T, None, T, None, T, None, g, None, g, need),
              (None, T, g, None, None, T, None, g, None, g, need), (None, T, g, T, None, None, None, g, None, g, need),
              (None, T, g, T, None, T, T, g, None, g, need), (d, T, g, T, None, T, None, g, None, g, need),
              (None, T, g, T, None, T, None, None, None, g, need), (None, T, g, T, None, T, None, g, odd, g, need),
              (None, T, g, T, None, T, None, g, None, None, need)):
        assert lib.upipe_layer_norm_bwd(c, *a, None) == -1
    assert lib.upipe_layer_norm_bwd(c, None, T, g, T, None, T, None, g, None, g, need - 1,
                                    None) == upipe.UPIPE_ERR_WS_TOO_SMALL
    assert upipe.launch_count() == n0


def test_binding_refuses_before_any_launch(lib):
    """Tensors on the CPU: nothing can run."""
    x, w = torch.zeros(4, 256, dtype=torch.bfloat16), torch.ones(256)
    W, t = torch.zeros(10, 256), torch.zeros(4, dtype=torch.int64)
    d = upipe.Dropout(0.1)
    n0 = upipe.launch_count()
    for f in (lambda: upipe.dropout_forward(d, x), lambda: upipe.dropout_forward(None, x),
              lambda: upipe.layer_norm_forward(x, w), lambda: upipe.layer_norm_forward(x[0], w),
              lambda: upipe.layer_norm_backward(x, w, x), lambda: upipe.layer_norm_fwd(x, w, None, x, s=x),
              lambda: upipe.embed_forward(t, W), lambda: upipe.embed_forward(t.float(), W),
              lambda: upipe.embed_forward(None, W), lambda: upipe.embed_forward(t, W.double()),
              lambda: upipe.embed_forward(t[None], W), lambda: upipe.embed_backward(t, x, 10),
              lambda: upipe.embed_backward(t, x[0], 10), lambda: upipe.dropout_apply(d, x, None, None)):
        with pytest.raises(ValueError):
            f()
    assert upipe.launch_count() == n0
    for n in (-1, 1 << 31, (1 << 32) + 256):
        assert upipe.layer_norm_workspace_bytes(4, n) == 0 and upipe.embed_workspace_bytes(n, 10, 256) == 0


def test_dropout_objects_check_and_copy_their_numbers():
    for bad in (dict(p=1.0), dict(p=-0.1), dict(p=float("nan")), dict(p=1 - 2.0 ** -33), dict(p=0.1, seed=-1),
                dict(p=0.1, seed=1 << 64), dict(p=0.1, call=1 << 64), dict(p=0.1, first=12), dict(p=0.1, first=-8), dict(p=0.1, first=1 << 63),
                dict(p=0.1, step=torch.zeros(1, dtype=torch.int64))):
        with pytest.raises(ValueError):
            upipe.Dropout(**bad)
    d = upipe.Dropout(0.25, seed=(1 << 64) - 1, call=1 << 63, first=64)
    for e in (copy.copy(d), copy.deepcopy(d), pickle.loads(pickle.dumps(d))):
        assert (e.p, e.seed, e.call, e.first, e.step) == (d.p, d.seed, d.call, d.first, None)
        assert e._c is not d._c and (e._c.seed, e._c.call) == (d.seed, d.call)
    with pytest.raises(AttributeError):
        d.call = 7


def test_descriptions_as_bytes_are_the_structures():
    """What the binding packs is what the mirrored structures hold, byte for byte
    (their padding apart from the values is zero in both)."""
    assert upipe._ROWS(1 << 40, 264, 0) == bytes(upipe.Rows(1 << 40, 264, 0))
    assert upipe._NORM(77, 1032, True, 1e-5) == bytes(upipe.NormCfg(77, 1032, 1, 1e-5))
    assert upipe._EMBED(9, 500, 64, True, False, 2.5) == bytes(upipe.EmbedCfg(9, 500, 64, 1, 0, 2.5))
