"""Rotary positions, query/key norms and windowed attention as they are used
together: a layer's heads through all three against the fp64 oracle, the
autograd front end against the binding's bits, a block that trains, a captured
training step, and the Ulysses chunk loop with a window."""

import os
import socket

import numpy as np
import pytest
import torch

from headwise_chunked_context_gb300 import synth, untied_ulysses as uu, upipe
from headwise_chunked_context_gb300.modules import QKNormRope, TiledCrossEntropy, TiledSwiGLU, rotate, window_attention
from oracle import local_oracle as loc
from tests.gpu_common import ensure_lib, f64, status_ok
from tests.tolerance import assert_close

pytestmark = pytest.mark.gpu

D128 = 128


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def _qkv(L, H, Hkv, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(L, H + 2 * Hkv, D128, generator=g, device="cuda").bfloat16()


@pytest.mark.parametrize("L,H,Hkv,W,S", [(1, 2, 1, 4, 1), (333, 4, 2, 100, 4), (700, 8, 2, 257, 130)])
def test_norm_rotation_and_window_together_match_the_oracle(L, H, Hkv, W, S):
    """Forward and gradients of the chain.  Each stage's output is rounded to
    bf16 (2^-8) before the next, so the oracle is fed the stage's own rounded
    inputs, and every stage is held to the attention core's tolerances."""
    qkv = _qkv(L, H, Hkv)
    q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:].contiguous()
    rope = upipe.Rope(D128, rot=64, layout="interleaved", scaling=("bands", 8.0, 1.0, 4.0, 8192))
    wq, wk = torch.linspace(0.8, 1.2, D128, device="cuda"), torch.linspace(1.1, 0.9, D128, device="cuda")
    pos = np.arange(L) + 5
    qr, kr = upipe.qk_norm_rope_forward(rope, q, k, wq, wk, pos0=5)
    cfg = upipe.WindowConfig(L=L, H=H, Hkv=Hkv, window=W, sinks=S)
    o, lse = upipe.window_forward(cfg, qr, kr, v)
    do = _qkv(L, H, 0, seed=1)
    dqr, dkr, dv = upipe.window_backward(cfg, qr, kr, v, o, lse, do)
    dq, dk, dwq, dwk = upipe.qk_norm_rope_backward(rope, q, k, wq, wk, dqr, dkr, pos0=5)
    status_ok()
    f = np.array(rope.freqs)
    args = (pos, f, 64, "interleaved")
    assert_close(f64(qr), loc.norm_rope(f64(q), f64(wq), 1e-6, *args), "q")
    assert_close(f64(kr), loc.norm_rope(f64(k), f64(wk), 1e-6, *args), "k")
    ro, rl = loc.window_fwd(f64(qr), f64(kr), f64(v), W, S)
    assert_close(f64(o), ro, "o")
    assert_close(f64(lse), rl, "lse")
    for got, want, n in zip((dqr, dkr, dv), loc.window_bwd(f64(qr), f64(kr), f64(v), f64(o), f64(do), W, S, True),
                            ("dq rotated", "dk rotated", "dv")):
        assert_close(f64(got), want, n)
    for x, w, dy, dx, dw, n in ((q, wq, dqr, dq, dwq, "q"), (k, wk, dkr, dk, dwk, "k")):
        rx, rw, _ = loc.norm_rope_bwd(f64(x), f64(w), 1e-6, f64(dy), *args)
        assert_close(f64(dx), rx, "d" + n)
        assert_close(f64(dw), rw, "dw" + n, weight_grad=True)


def test_functions_equal_the_binding():
    L, H, Hkv, W, S = 300, 4, 2, 70, 3
    rope = upipe.Rope(D128)
    qkv = _qkv(L, H, Hkv, 2).requires_grad_()
    m = QKNormRope(rope)
    with torch.no_grad():
        m.wq.copy_(torch.linspace(0.5, 1.5, D128))
    q, k = m(qkv[:, :H], qkv[:, H:H + Hkv], pos0=9)
    o = window_attention(q, k, qkv[:, H + Hkv:], W, S)
    do = _qkv(L, H, 0, 3)
    o.backward(do)
    x = qkv.detach()
    a = (x[:, :H].contiguous(), x[:, H:H + Hkv].contiguous(), x[:, H + Hkv:].contiguous())
    rq, rk = upipe.qk_norm_rope_forward(rope, *a[:2], m.wq.detach(), m.wk.detach(), pos0=9)
    cfg = upipe.WindowConfig(L=L, H=H, Hkv=Hkv, window=W, sinks=S)
    ro, lse = upipe.window_forward(cfg, rq, rk, a[2])
    dqr, dkr, dv = upipe.window_backward(cfg, rq, rk, a[2], ro, lse, do)
    dq, dk, dwq, dwk = upipe.qk_norm_rope_backward(rope, *a[:2], m.wq.detach(), m.wk.detach(), dqr, dkr, pos0=9)
    assert torch.equal(o, ro) and torch.equal(qkv.grad, torch.cat([dq, dk, dv], 1))
    assert torch.equal(m.wq.grad, dwq) and torch.equal(m.wk.grad, dwk)
    # rotation alone, with given positions and an expanded (broadcast) gradient
    pos = torch.randint(0, 1 << 20, (L,), dtype=torch.int32, device="cuda")
    q, k = a[0].clone().requires_grad_(), a[1].clone().requires_grad_()
    y, z = rotate(q, k, rope, positions=pos)
    (y.float().sum() + 2 * z.float().sum()).backward()
    gq, gk = upipe.rope_backward(rope, torch.ones_like(q), torch.full_like(k, 2.0), positions=pos)
    assert torch.equal(q.grad, gq) and torch.equal(k.grad, gk)
    status_ok()


def test_tensors_off_16_byte_boundaries_are_copied():
    """Dense, but one element into their storage, as gradients that come out
    of a concatenation are; and one token of rows whose length is no multiple
    of 8."""
    L, H, Hkv = 130, 4, 2

    def off(t):
        x = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape)
        return x.copy_(t)

    rope, qkv, do = upipe.Rope(D128), _qkv(L, H, Hkv, 4), _qkv(L, H, 0, 5)
    parts = [t.contiguous() for t in (qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:])]
    results = []
    for place in (torch.clone, off):
        q, k, v = (place(t).requires_grad_() for t in parts)
        m = QKNormRope(rope)
        a, b = m(q, k)
        o = window_attention(*(place(t) for t in rotate(a, b, rope, pos0=2)), place(v), 50, 3)
        o.backward(place(do))
        a, b = m(q, k)
        torch.autograd.backward(rotate(a, b, rope), (place(do), place(parts[1])))
        results.append((o, q.grad, k.grad, v.grad, m.wq.grad, m.wk.grad))
    assert off(parts[0]).data_ptr() % 16 and off(parts[0]).is_contiguous()
    assert all(torch.equal(x, y) for x, y in zip(*results))
    row = _qkv(1, 2, 0, 6).view(1, 256)
    x = torch.cat([row, row[:, :4]], 1).as_strided((1, 2, D128), (260, D128, 1))
    assert x.stride(0) % 8
    y, z = rotate(x, x, rope, pos0=7)
    assert torch.equal(y, rotate(row.view(1, 2, D128), row.view(1, 2, D128), rope, pos0=7)[0]) and torch.equal(y, z)
    status_ok()


def test_positions_changed_between_forward_and_backward_are_noticed():
    q, k = _qkv(8, 2, 0).requires_grad_(), _qkv(8, 1, 0).requires_grad_()
    rope = upipe.Rope(D128)
    for f in (lambda pos: rotate(q, k, rope, positions=pos), lambda pos: QKNormRope(rope)(q, k, positions=pos)):
        pos = torch.arange(8, dtype=torch.int32, device="cuda")
        y, _ = f(pos)
        pos += 1
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.float().sum().backward()
    status_ok()


def test_module_copies_and_second_derivatives_are_refused():
    import copy
    m = QKNormRope(upipe.Rope(D128, rot=64))
    qkv = _qkv(40, 2, 1, 8)
    a, b = m(qkv[:, :2], qkv[:, 2:3]), copy.deepcopy(m)(qkv[:, :2], qkv[:, 2:3])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    q, k, v = (t.contiguous().requires_grad_() for t in (qkv[:, :2], qkv[:, 2:3], qkv[:, 3:]))
    g = torch.autograd.grad(window_attention(q, k, v, 9, 1).float().square().sum(), q, create_graph=True)[0]
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.float().sum().backward()


def test_calls_from_a_thread_that_has_touched_no_device():
    """A fresh host thread has no current context; the library makes it
    current (autograd runs backwards on such threads)."""
    import threading
    q, k, v, do = (t.to("cuda:0") for t in synth.core_inputs(300, 4, 2))
    cfg, ccfg = upipe.WindowConfig(L=300, H=4, Hkv=2, window=70, sinks=3), upipe.Config(L=300, H=4, Hkv=2, U=4)
    o, lse = upipe.window_forward(cfg, q, k, v)
    co, clse = upipe.core_forward(ccfg, q, k, v)
    want = upipe.window_backward(cfg, q, k, v, o, lse, do) + upipe.core_backward(ccfg, q, k, v, co, clse, do)
    got = []

    def work(i):
        if i:
            got.append(upipe.core_backward(ccfg, q, k, v, co, clse, do))
        else:
            got.append(upipe.window_backward(cfg, q, k, v, o, lse, do))

    for i in range(2):
        t = threading.Thread(target=work, args=(i,))
        t.start()
        t.join()
    torch.cuda.synchronize()
    for a, b in zip(got[0] + got[1], want):
        assert torch.equal(a, b)
    status_ok()


class _Block(torch.nn.Module):
    """A layer with its own projections around the operators, an MLP and the loss."""

    def __init__(self, D=256, H=4, Hkv=2, F=512, V=512, window=100, sinks=4):
        super().__init__()
        self.H, self.Hkv, self.window, self.sinks = H, Hkv, window, sinks
        self.wqkv = torch.nn.Parameter(torch.randn((H + 2 * Hkv) * D128, D, device="cuda") * 0.05)
        self.wo = torch.nn.Parameter(torch.randn(D, H * D128, device="cuda") * 0.02)
        self.norm, self.mlp, self.ce = QKNormRope(upipe.Rope(D128)), TiledSwiGLU(D, F, 256), TiledCrossEntropy(D, V, 256)

    def hidden(self, x):
        qkv = (x @ self.wqkv.t().bfloat16()).view(x.shape[0], -1, D128)
        q, k = self.norm(qkv[:, :self.H], qkv[:, self.H:self.H + self.Hkv])
        o = window_attention(q, k, qkv[:, self.H + self.Hkv:], self.window, self.sinks)
        h = x + o.reshape(x.shape[0], -1) @ self.wo.t().bfloat16()
        return h + self.mlp(h)

    def forward(self, x, labels):
        return self.ce(self.hidden(x), labels)


def test_a_block_with_norm_rotation_and_window_has_gradients_everywhere():
    torch.manual_seed(4)
    m = _Block()
    x = torch.randn(500, 256, device="cuda").bfloat16().requires_grad_()
    labels = torch.randint(0, 512, (500,), device="cuda", dtype=torch.int32)
    m(x, labels).backward()
    for n, p in [*m.named_parameters(), ("x", x)]:
        assert p.grad is not None and torch.isfinite(p.grad).all() and p.grad.abs().max() > 0, n
    status_ok()


def test_captured_step_and_an_eager_call_beside_the_capture():
    """Forward and backward of the chain captured into one graph, replayed on
    new inputs; an eager backward on another stream between the captured
    call and the end of its capture does not join it."""
    L, H, Hkv = 300, 4, 2
    rope, w = upipe.Rope(D128), torch.ones(D128, device="cuda")
    cfg = upipe.WindowConfig(L=L, H=H, Hkv=Hkv, window=80, sinks=2)

    def step(qkv, do):
        q, k = upipe.qk_norm_rope_forward(rope, qkv[:, :H], qkv[:, H:H + Hkv], w, w)
        v = qkv[:, H + Hkv:].contiguous()
        o, lse = upipe.window_forward(cfg, q, k, v)
        dq, dk, dv = upipe.window_backward(cfg, q, k, v, o, lse, do)
        return (o, dv, *upipe.qk_norm_rope_backward(rope, qkv[:, :H], qkv[:, H:H + Hkv], w, w, dq, dk))

    qkv, do = _qkv(L, H, Hkv, 5), _qkv(L, H, 0, 6)
    want = step(qkv, do)  # first call outside capture
    q, k, v = (qkv[:, :H].contiguous(), qkv[:, H:H + Hkv].contiguous(), qkv[:, H + Hkv:].contiguous())
    o, lse = upipe.window_forward(cfg, q, k, v)
    eager = upipe.window_backward(cfg, q, k, v, o, lse, do)
    out = [torch.zeros_like(t) for t in eager]
    ws = torch.empty(upipe.window_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, capture_error_mode="relaxed"):
        got = step(qkv, do)
        upipe.window_bwd(cfg, q, k, v, o, lse, do, *out, ws=ws, stream=other)  # not captured: runs now
    torch.cuda.synchronize()
    for a, b in zip(out, eager):
        assert torch.equal(a, b)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    qkv.copy_(_qkv(L, H, Hkv, 7))
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, step(qkv, do)):
        assert torch.equal(a, b)
    status_ok()


@pytest.mark.parametrize("L,H,Hkv,U,P", [(1024, 8, 2, 4, 2), (512, 16, 2, 8, 2)])
def test_rank_rows_rotated_before_the_exchange(L, H, Hkv, U, P):
    """A rank's rows, rotated with its first row as pos0, are the rows of the
    whole sequence rotated at once: the sequence-sharded input of the loop."""
    q, k, _, _ = (t.to("cuda:0") for t in synth.core_inputs(L, H, Hkv))
    rope = upipe.Rope(D128)
    want = upipe.rope_forward(rope, q, k)
    for r in range(P):
        rows = slice(uu.rows_of(L, P, r)[0], uu.rows_of(L, P, r)[-1] + 1)
        got = upipe.rope_forward(rope, q[rows], k[rows], pos0=rows.start)
        assert torch.equal(got[0], want[0][rows]) and torch.equal(got[1], want[1][rows])


@pytest.mark.parametrize("L,H,Hkv,U", [(1024, 8, 2, 4), (512, 8, 2, 2)])
def test_chunk_loop_with_a_window_on_one_nccl_rank(L, H, Hkv, U):
    """untied_ulysses.forward / backward with gpu_core(window, sinks): the
    windowed attention's O, LSE and dQ bits; dK / dV too for U >= g, within
    the tolerance for U < g (a KV head's chunk partials are summed)."""
    import torch.distributed as dist
    with socket.socket() as sk:
        sk.bind(("127.0.0.1", 0))
        port = sk.getsockname()[1]
    os.environ["MASTER_ADDR"] = "127.0.0.1"
    os.environ["MASTER_PORT"] = str(port)
    dist.init_process_group("nccl", rank=0, world_size=1, device_id=torch.device("cuda:0"))
    try:
        q, k, v, do = (t.to("cuda:0") for t in synth.core_inputs(L, H, Hkv))
        core_fwd, core_bwd = uu.gpu_core(window=200, sinks=4)
        o, lse = uu.forward(q, k, v, H, Hkv, U, core_fwd)
        dq, dk, dv = uu.backward(q, k, v, o, lse, do, H, Hkv, U, core_bwd)
        cfg = upipe.WindowConfig(L=L, H=H, Hkv=Hkv, window=200, sinks=4)
        ro, rlse = upipe.window_forward(cfg, q, k, v)
        rdq, rdk, rdv = upipe.window_backward(cfg, q, k, v, ro, rlse, do)
        torch.cuda.synchronize()
        status_ok()
        assert torch.equal(o, ro) and torch.equal(dq, rdq)
        for c in uu.plan(H, Hkv, U, 1):
            assert torch.equal(lse[c.c], rlse[list(c.q_heads[0])])
        if U >= H // Hkv:
            assert torch.equal(dk.bfloat16(), rdk) and torch.equal(dv.bfloat16(), rdv)
        else:
            assert_close(f64(dk), f64(rdk), "dk (chunk partials summed in fp32)")
            assert_close(f64(dv), f64(rdv), "dv (chunk partials summed in fp32)")
    finally:
        dist.destroy_process_group()


def test_norm_module_with_weights_of_another_type():
    """QKNormRope after .bfloat16(), as the package's other modules run:
    computed with the fp32 value of each weight, gradients in the weight's type."""
    rope, qkv = upipe.Rope(D128), _qkv(60, 3, 2, 9)
    q, k = qkv[:, :3], qkv[:, 3:5]
    m = QKNormRope(rope).bfloat16()
    with torch.no_grad():
        m.wq.copy_(torch.linspace(0.5, 1.5, D128))
    y = m(q, k)
    w = (m.wq.detach().float(), m.wk.detach().float())
    for a, b in zip(y, upipe.qk_norm_rope_forward(rope, q, k, *w)):
        assert torch.equal(a, b)
    dq, dk = _qkv(60, 3, 0, 10), _qkv(60, 2, 0, 11)
    torch.autograd.backward(y, (dq, dk))
    want = upipe.qk_norm_rope_backward(rope, q, k, *w, dq, dk)[2:]
    assert m.wq.dtype == m.wq.grad.dtype == torch.bfloat16
    assert torch.equal(m.wq.grad, want[0].bfloat16()) and torch.equal(m.wk.grad, want[1].bfloat16())
    status_ok()


def test_captured_training_step_of_the_modules():
    """Forward and backward of norm, rotation and window through autograd,
    captured after a warm-up on a side stream and replayed on new inputs."""
    L, H, Hkv = 260, 4, 2
    m, rope = QKNormRope(upipe.Rope(D128, rot=64)), upipe.Rope(D128, layout="interleaved")
    with torch.no_grad():
        m.wk.copy_(torch.linspace(0.5, 1.5, D128))
    qkv, do = _qkv(L, H, Hkv, 12).requires_grad_(), _qkv(L, H, 0, 13)
    leaves = (qkv, m.wq, m.wk)

    def step():
        q, k = m(qkv[:, :H], qkv[:, H:H + Hkv])
        o = window_attention(*rotate(q, k, rope, pos0=3), qkv[:, H + Hkv:], 60, 2)
        return (o, *torch.autograd.grad(o, leaves, do))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (14, 15):
        with torch.no_grad():
            qkv.copy_(_qkv(L, H, Hkv, seed))
        do.copy_(_qkv(L, H, 0, seed + 10))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
    status_ok()
