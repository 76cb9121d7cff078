"""GPU parity of windowed attention with sinks against the fp64 oracle: the
tolerances of the attention core (tests/tolerance.py), against the precision
model (P and dS enter their products as bf16) and the plain definition; and
masks read back exactly from uniform scores."""

import numpy as np
import pytest
import torch

from headwise_chunked_context_gb300 import synth, upipe
from oracle import local_oracle as loc
from tests.gpu_common import dev, ensure_lib, f64, status_ok
from tests.tolerance import assert_close, assert_close_plain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


# L, H, Hkv, window, sinks: one token, windows of one key, inside a tile, of whole tiles, one more or
# less, past the sequence; sinks of none, one, part of a tile, whole tiles, more than the sequence
CASES = [
    (1, 1, 1, 1, 0), (1, 2, 1, 5, 3), (2, 1, 1, 1, 1), (127, 2, 1, 1, 0), (128, 4, 2, 128, 0), (129, 4, 1, 64, 4),
    (300, 4, 1, 100, 4), (300, 2, 2, 300, 0), (257, 2, 1, 2, 1), (385, 4, 2, 129, 1), (640, 2, 1, 127, 130),
    (640, 2, 1, 128, 128), (641, 2, 1, 1, 640), (1000, 4, 1, 257, 5), (1000, 2, 1, 1, 1), (700, 2, 1, 2000, 3),
    (500, 2, 1, 40, 9000), (1100, 8, 2, 200, 300), (1500, 4, 4, 513, 16), (2049, 2, 1, 129, 1),
    (1300, 2, 1, 900, 700), (1300, 4, 2, 640, 1000), (3000, 2, 1, 1, 130), (2200, 1, 1, 300, 2100),
]


def _run(L, H, Hkv, W, S, seed_shift=0):
    q, k, v, do = synth.core_inputs(L, H, Hkv)
    cfg = upipe.WindowConfig(L=L, H=H, Hkv=Hkv, window=W, sinks=S)
    qd, kd, vd, dod = dev(q, k, v, do)
    o, lse = upipe.window_forward(cfg, qd, kd, vd)
    grads = upipe.window_backward(cfg, qd, kd, vd, o, lse, dod)
    torch.cuda.synchronize()
    status_ok()
    return (q, k, v, do), (o, lse, *grads)


@pytest.mark.parametrize("L,H,Hkv,W,S", CASES)
def test_window_matches_oracle(L, H, Hkv, W, S):
    (q, k, v, do), got = _run(L, H, Hkv, W, S)
    q, k, v, do = (f64(t) for t in (q, k, v, do))
    o, lse = loc.window_fwd(q, k, v, W, S)
    # The backward is a function of the o it is given, so the model gets the same one.  With the exact o
    # instead, Delta = sum_c dO_c o_c would be off by the given o's own error, 128^.5 * 2^-8 |o| (P and o are
    # rounded to bf16), 0.03 for o of 0.7; a sink's dK adds that up over every query: P 0.03 |q| / 128^.5 n^.5,
    # 0.02 for n = 514 queries with P = 1/3, 0.06 at the largest of 128 columns (3 sigma), past the 0.02.
    model = (o, lse, *loc.window_bwd(q, k, v, f64(got[0]), do, W, S, bf16_operands=True))
    plain = (o, lse, *loc.window_bwd(q, k, v, o, do, W, S))
    for a, m, p, n in zip(got, model, plain, ("o", "lse", "dq", "dk", "dv")):
        assert_close(f64(a), m, n)
        assert_close_plain(f64(a), p, m, n)


@pytest.mark.parametrize("L,W,S", [(1, 1, 0), (300, 1, 0), (300, 100, 4), (640, 128, 0), (640, 129, 128),
                                   (641, 127, 129), (900, 256, 300), (2500, 700, 200), (2500, 5000, 0)])
def test_window_visits_exactly_the_visible_keys(L, W, S):
    """Scores are all zero and key j's value is 1 in column j % 128: row i of O
    is the count of visible keys per column over their number n.  P is 2^0
    and the count is exact; O is rounded to bf16 (2^-8 of it) after one fp32
    division (1e-6).  LSE is ln n.  One key too many or too few changes a
    column by at least 1 / 20 of it here."""
    q = torch.zeros(L, 2, 128, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(L, 1, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros(L, 1, 128, dtype=torch.bfloat16, device="cuda")
    v[torch.arange(L), 0, torch.arange(L) % 128] = 1.0
    cfg = upipe.WindowConfig(L=L, H=2, Hkv=1, window=W, sinks=S)
    o, lse = upipe.window_forward(cfg, q, k, v)
    seen = loc.visible(np.arange(L), np.arange(L), W, S)
    n = seen.sum(1)
    want = (seen @ f64(v)[:, 0]) / n[:, None]
    for h in range(2):
        assert np.all(np.abs(f64(o)[:, h] - want) <= (2.0 ** -8 + 1e-6) * want)
        np.testing.assert_allclose(f64(lse)[h], np.log(n), rtol=0, atol=2e-6)
    # dV of a dO of ones in one column: sum over the queries that see key j of 1/n_i.  P is rounded to
    # bf16 (2^-8), the sum over at most 2500 queries in fp32, dV to bf16 (2^-8).
    do = torch.zeros_like(q)
    do[:, :, 5] = 1.0
    dq, dk, dv = upipe.window_backward(cfg, q, k, v, o, lse, do)
    want = 2 * (seen / n[:, None]).sum(0)
    assert np.all(np.abs(f64(dv)[:, 0, 5] - want) <= (2 * 2.0 ** -8 + 1e-4) * want)
    assert not dq.any() and not dk.any()  # k and q are zero
    status_ok()


def test_window_past_the_sequence_is_the_causal_core():
    q, k, v, do = dev(*synth.core_inputs(777, 4, 2))
    cfg = upipe.Config(L=777, H=4, Hkv=2, U=4)
    o, lse = upipe.core_forward(cfg, q, k, v)
    want = (o, lse, *upipe.core_backward(cfg, q, k, v, o, lse, do))
    for W, S in ((777, 0), (10 ** 12, 0), (5, 10 ** 12)):
        wc = upipe.WindowConfig(L=777, H=4, Hkv=2, window=W, sinks=S)
        o, lse = upipe.window_forward(wc, q, k, v)
        for a, b, n in zip((o, lse, *upipe.window_backward(wc, q, k, v, o, lse, do)), want,
                           ("o", "lse", "dq", "dk", "dv")):
            assert_close(f64(a), f64(b), n)


def test_window_large_scores_and_the_same_bits_again():
    """Scores of some hundreds: the running maximum moves, rows keep one key."""
    L, H, Hkv, W, S = 520, 2, 1, 150, 2
    q, k, v, do = synth.core_inputs(L, H, Hkv)
    q = (q.float() * 16).bfloat16()
    cfg = upipe.WindowConfig(L=L, H=H, Hkv=Hkv, window=W, sinks=S)
    qd, kd, vd, dod = dev(q, k, v, do)
    runs = []
    for _ in range(2):
        o, lse = upipe.window_forward(cfg, qd, kd, vd)
        runs.append((o, lse, *upipe.window_backward(cfg, qd, kd, vd, o, lse, dod)))
    for a, b in zip(*runs):
        assert torch.equal(a, b)
    ro, rl = loc.window_fwd(f64(q), f64(k), f64(v), W, S)
    assert_close(f64(runs[0][0]), ro, "o")
    np.testing.assert_allclose(f64(runs[0][1]), rl, rtol=1e-5, atol=1e-4)
    status_ok()


@pytest.mark.parametrize("L,H,Hkv,W,S", [(2200, 1, 1, 300, 2100), (1300, 4, 2, 640, 1000), (20000, 2, 2, 1, 0),
                                         (9000, 4, 1, 130, 140)])
def test_window_many_short_items_give_the_same_bits_every_time(L, H, Hkv, W, S):
    """More tiles and key items than CTAs, of one or two blocks each, so that
    loads, products and epilogues of neighbouring items overlap: nothing that
    a product reads may still be on its way, or be overwritten early."""
    q, k, v, do = dev(*synth.core_inputs(L, H, Hkv))
    cfg = upipe.WindowConfig(L=L, H=H, Hkv=Hkv, window=W, sinks=S)
    want = None
    for _ in range(25):
        o, lse = upipe.window_forward(cfg, q, k, v)
        got = (o, lse, *upipe.window_backward(cfg, q, k, v, o, lse, do))
        want = want or got
        for a, b, n in zip(got, want, ("o", "lse", "dq", "dk", "dv")):
            assert torch.equal(a, b), n
    if W == 1:  # each query sees itself alone
        assert torch.equal(want[0], v.repeat_interleave(H // Hkv, 1)) and torch.equal(want[4], do)
    status_ok()


def test_window_on_another_stream_and_captured():
    L, H, Hkv = 400, 4, 2
    q, k, v, do = dev(*synth.core_inputs(L, H, Hkv))
    cfg = upipe.WindowConfig(L=L, H=H, Hkv=Hkv, window=90, sinks=3)
    o, lse = upipe.window_forward(cfg, q, k, v)
    want = (o, lse, *upipe.window_backward(cfg, q, k, v, o, lse, do))
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    out = [torch.empty_like(t) for t in want]
    upipe.window_fwd(cfg, q, k, v, out[0], out[1], stream=st)
    upipe.window_bwd(cfg, q, k, v, out[0], out[1], do, *out[2:], stream=st)
    st.synchronize()
    for a, b in zip(out, want):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o2, lse2 = upipe.window_forward(cfg, q, k, v)
        got = (o2, lse2, *upipe.window_backward(cfg, q, k, v, o2, lse2, do))
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    status_ok()


def test_window_writes_nothing_past_its_rows():
    """Rows behind the last token, in the same allocation, stay as they were."""
    L, H, Hkv = 130, 2, 1
    q, k, v, do = dev(*synth.core_inputs(L, H, Hkv))
    cfg = upipe.WindowConfig(L=L, H=H, Hkv=Hkv, window=50, sinks=2)
    big = {n: torch.full((L + 200, h, 128), 7.0, dtype=torch.bfloat16, device="cuda")
           for n, h in (("o", H), ("dq", H), ("dk", Hkv), ("dv", Hkv))}
    lse = torch.full((H * L + 500,), 7.0, device="cuda")
    upipe.window_fwd(cfg, q, k, v, big["o"][:L], lse[:H * L].view(H, L))
    upipe.window_bwd(cfg, q, k, v, big["o"][:L], lse[:H * L].view(H, L), do, big["dq"][:L], big["dk"][:L],
                     big["dv"][:L])
    torch.cuda.synchronize()
    for t in big.values():
        assert bool((t[L:] == 7.0).all())
    assert bool((lse[H * L:] == 7.0).all())
    status_ok()


def test_window_workspace_refusal():
    L, H, Hkv = 64, 2, 1
    q, k, v, do = dev(*synth.core_inputs(L, H, Hkv))
    cfg = upipe.WindowConfig(L=L, H=H, Hkv=Hkv, window=5)
    o, lse = upipe.window_forward(cfg, q, k, v)
    need = upipe.window_workspace_bytes(cfg)
    with pytest.raises(ValueError, match="ws"):
        upipe.window_bwd(cfg, q, k, v, o, lse, do, q.clone(), k.clone(), v.clone(),
                         ws=torch.empty(need - 16, dtype=torch.uint8, device="cuda"))


def test_window_outputs_on_16_byte_boundaries_have_the_same_bits():
    """Outputs 16 bytes past a 32-byte boundary are stored in halves of it;
    the 16 bytes before and after them stay as they were."""
    L, H, Hkv = 300, 4, 2
    q, k, v, do = dev(*synth.core_inputs(L, H, Hkv))
    cfg = upipe.WindowConfig(L=L, H=H, Hkv=Hkv, window=90, sinks=5)
    o, lse = upipe.window_forward(cfg, q, k, v)
    grads = upipe.window_backward(cfg, q, k, v, o, lse, do)

    def off(heads):
        room = torch.full((L * heads * 128 + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
        return room, room[8:-8].view(L, heads, 128)

    rooms, (o2, dq, dk, dv) = zip(*(off(n) for n in (H, H, Hkv, Hkv)))
    assert all(t.data_ptr() % 32 == 16 for t in (o2, dq, dk, dv))
    lse2 = torch.empty_like(lse)
    upipe.window_fwd(cfg, q, k, v, o2, lse2)
    upipe.window_bwd(cfg, q, k, v, o2, lse2, do, dq, dk, dv)
    status_ok()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    for a, b in zip(grads, (dq, dk, dv)):
        assert torch.equal(a, b)
    for room in rooms:
        assert (room[:8] == 7).all() and (room[-8:] == 7).all()


@pytest.mark.parametrize("L,H,Hkv,W,S,loud", [(520, 2, 1, 150, 2, 1), (520, 2, 1, 150, 2, 8), (1100, 4, 2, 64, 130, 8),
                                              (300, 4, 1, 300, 0, 8), (700, 2, 2, 1, 3, 8)])
def test_window_gradients_at_large_scores(L, H, Hkv, W, S, loud):
    """Scores of tens to hundreds against the plain definition (with the given
    o in Delta, see test_window_matches_oracle), and hidden keys, before the
    window and after the query, whose exponentials overflow.  Element by
    element, with b = 2^-8 for each rounding to bf16:
    S: sums of 128 products and -LSE in fp32, each of 10 steps off by at most
    2^-23 of the largest partial sum; LSE comes from such scores too, so P is
    off by e_i = 20 2^-23 (max_j sum_c |q_c k_c| / sqrt(d) + |LSE_i|) + 4e-6 of
    itself (the last for exp2 and log2 in fp32).
    dP - Delta: off by n_ij = 12 2^-23 sum_c |dO_c| (|v_c| + |o_c|).
    dS enters its products with an error of P (|dP - Delta| (e + b) + n), P
    with P (e + b); the products' sums over at most 70 steps add 70 2^-23 of
    their terms' sizes, and each output is rounded to bf16 once."""
    q, k, v, do = synth.core_inputs(L, H, Hkv)
    q, k = (q.float() * 16).bfloat16(), k.clone()
    k[13::97] *= loud
    cfg = upipe.WindowConfig(L=L, H=H, Hkv=Hkv, window=W, sinks=S)
    qd, kd, vd, dod = dev(q, k, v, do)
    o, lse = upipe.window_forward(cfg, qd, kd, vd)
    got = [f64(t) for t in (o, *upipe.window_backward(cfg, qd, kd, vd, o, lse, dod))]
    status_ok()
    q, k, v, do = (f64(t) for t in (q, k, v, do))
    seen, g, rt = loc.visible(np.arange(L), np.arange(L), W, S), H // Hkv, 128 ** 0.5
    b, add = 2.0 ** -8, 70 * 2.0 ** -23
    want = [np.zeros_like(x) for x in got]
    slack = [np.zeros_like(x) for x in got]
    above = 0.0
    for h in range(H):
        kv = h // g
        s = q[:, h] @ k[:, kv].T / rt
        m = np.where(seen, s, -np.inf).max(1)
        ref = m + np.log(np.exp(np.where(seen, s, -np.inf) - m[:, None]).sum(1))
        above = max(above, np.max(np.where(seen, -np.inf, s) - ref[:, None]))
        size = (np.abs(q[:, h]) @ np.abs(k[:, kv]).T / rt * seen).max(1)
        e = (20 * 2.0 ** -23 * (size + np.abs(ref)) + 4e-6)[:, None]
        assert np.all(np.abs(f64(lse)[h] - ref) <= e[:, 0])
        p = np.where(seen, np.exp(np.where(seen, s, -np.inf) - ref[:, None]), 0.0)
        d = do[:, h] @ v[:, kv].T - np.sum(do[:, h] * got[0][:, h], 1, keepdims=True)
        n = 12 * 2.0 ** -23 * (np.abs(do[:, h]) @ np.abs(v[:, kv]).T +
                               np.sum(np.abs(do[:, h] * got[0][:, h]), 1, keepdims=True))
        ds, dserr, perr = p * d, p * (np.abs(d) * (e + b + add) + n), p * (e + b + add)
        for i, head, value, err, x, scale in ((0, h, p, perr, v[:, kv], 1.0), (1, h, ds, dserr, k[:, kv], rt),
                                              (2, kv, ds.T, dserr.T, q[:, h], rt), (3, kv, p.T, perr.T, do[:, h], 1.0)):
            want[i][:, head] += value @ x / scale
            slack[i][:, head] += err @ np.abs(x) / scale
    assert loud == 1 or above > 100  # exp of it is past fp32
    for a, w, t, name in zip(got, want, slack, ("o", "dq", "dk", "dv")):
        over = np.abs(a - w) - (t * (1 + b) + b * np.abs(w) + 1e-30)
        at = np.unravel_index(over.argmax(), over.shape)
        assert np.isfinite(a).all() and over.max() <= 0, f"{name}: {over.max():.3e} over at {at}"
