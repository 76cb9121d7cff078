"""Token embedding, dropout and norms as they are used together: a chain of
them with the MLP and the loss against the fp64 oracles, the autograd front end
against the binding's bits, a small model with gradients everywhere,
recomputation, captured training steps and a tied table."""

import copy
import threading

import numpy as np
import pytest
import torch
from torch.utils.checkpoint import checkpoint

from headwise_chunked_context_gb300 import upipe
from headwise_chunked_context_gb300.modules import (HeadChunkedAttention, LayerNorm, TiledCrossEntropy, TiledSwiGLU,
                                                    TokenEmbedding, dropout)
from oracle import residual_oracle as res
from tests.gpu_common import ensure_lib, f64, status_ok
from tests.tolerance import assert_close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def _randn(seed, *shape, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).bfloat16()


def _tokens(seed, L, V, pad=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.randint(0, V, (L,), generator=g, device="cuda")
    t[-pad:] = -1
    return t


@pytest.mark.parametrize("L,D,rms,p", [(130, 256, True, 0.1), (257, 384, False, 0.5), (5, 128, False, 0.0)])
def test_embedding_norms_mlp_and_loss_together_match_the_oracles(L, D, rms, p):
    """tokens -> embedding -> dropout -> norm -> MLP -> dropout, sum, norm ->
    loss, and back to the table's gradient.  Each stage's output is rounded to
    bf16 before the next, so every oracle is fed its stage's own inputs and every
    stage is held to the package's tolerances."""
    V, F, T = 512, 256, 128
    tokens, labels = _tokens(0, L, V), _tokens(1, L, V).int()
    table, wgu, wd, head = (_randn(i, *s, std=0.05) for i, s in ((2, (V, D)), (3, (2 * F, D)), (4, (D, F)), (5, (V, D))))
    w1, b1 = 1 + 0.1 * _randn(6, D).float(), 0.1 * _randn(7, D).float()
    w2, b2 = 1 + 0.1 * _randn(8, D).float(), 0.1 * _randn(9, D).float()
    d0, d1 = dict(p=p, seed=11, call=0), dict(p=p, seed=11, call=1)
    kw = dict(eps=1e-5, rms=rms)
    scale = D ** 0.5
    e = upipe.embed_forward(tokens, table.float(), scale)
    s0 = upipe.dropout_forward(upipe.Dropout(**d0), e)
    y0, _ = upipe.layer_norm_forward(s0, w1, b1, **kw)
    m = upipe.mlp_forward(y0, wgu, wd, T)
    y1, s1 = upipe.layer_norm_forward(m, w2, b2, residual=s0, dropout=upipe.Dropout(**d1), **kw)
    lscale = 1.0 / max(1, int((labels >= 0).sum()))
    loss, dy1, dhead = upipe.ce_loss(y1, head, labels, lscale, T)
    dm, ds0, dw2, db2 = upipe.layer_norm_backward(s1, w2, dy1, dropout=upipe.Dropout(**d1), **kw)
    dy0, dwgu, dwd = upipe.mlp_backward(y0, wgu, wd, dm, T)
    dsum, dres, dw1, db1 = upipe.layer_norm_backward(s0, w1, dy0, ds0, **kw)
    assert dsum is dres
    de = upipe.dropout_backward(upipe.Dropout(**d0), dsum)
    dtable = upipe.embed_backward(tokens, de, V, scale)
    status_ok()
    t = tokens.cpu().numpy()
    assert_close(f64(e), res.embed(t, f64(table), float(np.float32(scale))), "embedding")
    assert_close(f64(s0), res.drop(f64(e), **d0), "dropout")
    assert_close(f64(y0), res.norm(f64(s0), f64(w1), f64(b1), 1e-5, rms), "norm")
    assert_close(f64(s1), res.add(f64(m), f64(s0), **d1), "sum")
    assert_close(f64(y1), res.norm(f64(s1), f64(w2), f64(b2), 1e-5, rms), "norm of the sum")
    g, gw, gb = res.norm_bwd(f64(s1), f64(w2), f64(dy1), None, 1e-5, rms)
    # the loss's gradients are small: the tolerances are of numbers around one
    big = 1.0 / max(1e-30, float(np.abs(g).max()))
    assert_close(big * f64(ds0), big * g, "gradient of the sum")
    assert_close(big * f64(dm), big * res.drop(g, **d1), "gradient behind the mask")
    assert_close(big * f64(dw2), big * gw, "dw2", weight_grad=True)
    assert_close(big * f64(db2), big * gb, "db2", weight_grad=True)
    g, gw, gb = res.norm_bwd(f64(s0), f64(w1), f64(dy0), f64(ds0), 1e-5, rms)
    big = 1.0 / max(1e-30, float(np.abs(g).max()))
    assert_close(big * f64(dsum), big * g, "gradient of the stream")
    assert_close(big * f64(dw1), big * gw, "dw1", weight_grad=True)
    assert_close(big * f64(db1), big * gb, "db1", weight_grad=True)
    assert_close(big * f64(de), big * res.drop(f64(dsum), **d0), "gradient of the embedding")
    want = res.embed_bwd(t, f64(de), V, float(np.float32(scale)))[0]
    assert_close(big * f64(dtable), big * want, "table", weight_grad=True)
    assert np.isfinite(f64(loss)).all()


def test_functions_equal_the_binding():
    L, V, D = 200, 90, 264
    tokens = _tokens(20, L, V)
    emb = TokenEmbedding(V, D, scale=3.0)
    y = emb(tokens)
    assert torch.equal(y, upipe.embed_forward(tokens, emb.w.detach(), 3.0))
    dy = _randn(21, L, D)
    y.backward(dy)
    assert torch.equal(emb.w.grad, upipe.embed_backward(tokens, dy, V, 3.0))
    # dropout, with and without a residual, and none at all
    d = upipe.Dropout(0.3, seed=5, call=2)
    x, r = _randn(22, L, D).requires_grad_(), _randn(23, L, D).requires_grad_()
    y = dropout(x, d, r)
    assert torch.equal(y, upipe.dropout_forward(d, x.detach(), r.detach()))
    y.backward(dy)
    assert torch.equal(x.grad, upipe.dropout_backward(d, dy)) and torch.equal(r.grad, dy)
    x.grad = None
    dropout(x, d).backward(dy)
    assert torch.equal(x.grad, upipe.dropout_backward(d, dy))
    assert dropout(x, None) is x
    assert torch.equal(dropout(x, None, r), (r.detach().float() + x.detach().float()).bfloat16())
    # norms: alone, behind a sum, behind a mask
    for rms in (False, True):
        m = LayerNorm(D, eps=1e-4, rms=rms)
        assert (m.b is None) == rms
        with torch.no_grad():
            m.w.copy_(torch.linspace(0.5, 1.5, D))
        b = None if rms else m.b.detach()
        kw = dict(eps=1e-4, rms=rms)
        for residual, drop in ((None, None), (r, None), (r, d), (None, d)):
            for t in (x, r, m.w, m.b):
                if t is not None:
                    t.grad = None
            out = m(x, residual, drop)
            want = upipe.layer_norm_forward(x.detach(), m.w.detach(), b, residual=None if residual is None else r.detach(),
                                            dropout=drop, **kw)
            ds = None
            if residual is None and drop is None:
                assert torch.equal(out, want[0])
                out.backward(dy)
            else:
                assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
                ds = _randn(24, L, D)
                torch.autograd.backward(out, (dy, ds))
            dx, dres, dw, db = upipe.layer_norm_backward(want[1], m.w.detach(), dy, ds, bias=not rms, dropout=drop, **kw)
            assert torch.equal(x.grad, dx) and torch.equal(m.w.grad, dw)
            assert rms or torch.equal(m.b.grad, db)
            assert residual is None or torch.equal(r.grad, dres)
    status_ok()


def test_parts_of_a_norms_outputs_that_nothing_uses():
    """Only the norm, only the sum behind it, and gradients that are one row for all."""
    L, D = 60, 256
    x, r, dy = _randn(30, L, D).requires_grad_(), _randn(31, L, D).requires_grad_(), _randn(32, L, D)
    m, d = LayerNorm(D), upipe.Dropout(0.4, seed=9)
    y, s = m(x, r, d)
    gx, gr, gw = torch.autograd.grad(y, (x, r, m.w), dy, retain_graph=True)
    want = upipe.layer_norm_backward(s.detach(), m.w.detach(), dy, dropout=d)
    assert torch.equal(gx, want[0]) and torch.equal(gr, want[1]) and torch.equal(gw, want[2])
    gx, gr, gw, gb = torch.autograd.grad(s, (x, r, m.w, m.b), dy)
    assert torch.equal(gx, upipe.dropout_backward(d, dy)) and torch.equal(gr, dy)
    assert not gw.any() and not gb.any()
    y, s = m(x, r.detach())  # a residual without a gradient
    (y.float().sum() + s.float().sum()).backward()
    one = torch.ones_like(dy)
    want = upipe.layer_norm_backward(s.detach(), m.w.detach(), one, one)
    assert torch.equal(x.grad, want[0]) and r.grad is None
    t = _tokens(33, L, 20)
    emb = TokenEmbedding(20, D)
    emb(t).float().sum().backward()
    assert torch.equal(emb.w.grad, upipe.embed_backward(t, one, 20))


def test_tensors_off_16_byte_boundaries_and_of_other_types_are_copied():
    L, D = 50, 264

    def off(t):
        return torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape).copy_(t)

    d, dy = upipe.Dropout(0.2, seed=1), _randn(40, L, D)
    results = []
    for place in (torch.clone, off, lambda t: t.float(), lambda t: t.t().contiguous().t()):
        x, r = place(_randn(41, L, D)).requires_grad_(), place(_randn(42, L, D)).requires_grad_()
        m = LayerNorm(D)
        y, s = m(x, r, d)
        z = dropout(s, d, y)
        z.backward(off(dy))
        results.append((z, x.grad.bfloat16(), r.grad.bfloat16(), m.w.grad, m.b.grad))
    for other in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(results[0], other))
    # modules of another type compute with the fp32 value of each weight
    m = LayerNorm(D).bfloat16()
    x = _randn(43, L, D)
    y = m(x)
    y.backward(dy)
    want = upipe.layer_norm_backward(x, m.w.detach().float(), dy)
    assert m.w.grad.dtype == torch.bfloat16 and torch.equal(m.w.grad, want[2].bfloat16())
    for dtype in (torch.bfloat16, torch.float64):
        emb = TokenEmbedding(30, D).to(dtype)
        t = _tokens(44, L, 30).to(torch.int16).long()
        y = emb(t.int())
        y.backward(dy)
        assert torch.equal(y, upipe.embed_forward(t, emb.w.detach().float())) and emb.w.grad.dtype == dtype
        assert torch.equal(emb.w.grad, upipe.embed_backward(t, dy, 30).to(dtype))
    status_ok()


def test_a_step_or_a_stream_changed_before_the_backward_is_noticed():
    L, D = 20, 256
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    d, m = upipe.Dropout(0.2, seed=1, step=step), LayerNorm(D)
    x = _randn(50, L, D).requires_grad_()
    for f in (lambda: dropout(x, d), lambda: m(x, None, d)[0]):
        y = f()
        step += 1
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.float().sum().backward()
    y, s = m(x, x)
    s += 1
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.float().sum().backward()


def test_copies_and_second_derivatives():
    D = 256
    m, x = LayerNorm(D), _randn(60, 30, D).requires_grad_()
    assert torch.equal(copy.deepcopy(m)(x), m(x))
    emb = TokenEmbedding(40, D)
    t = _tokens(61, 30, 40)
    assert torch.equal(copy.deepcopy(emb)(t), emb(t))
    d = upipe.Dropout(0.5, seed=3, call=4)
    assert torch.equal(dropout(x, copy.deepcopy(d)), dropout(x, d))
    for f in (lambda: m(x), lambda: dropout(x, d)):
        g = torch.autograd.grad(f().float().square().sum(), x, create_graph=True)[0]
        with pytest.raises(RuntimeError, match="once_differentiable"):
            g.float().sum().backward()


class _Model(torch.nn.Module):
    """Embedding, one block of attention and MLP, and the loss; the masks of a
    step are numbers of (seed, step)."""

    def __init__(self, V=512, D=256, H=4, Hkv=2, U=2, F=512, rms=True):
        super().__init__()
        self.emb = TokenEmbedding(V, D, scale=D ** 0.5)
        self.n1, self.n2, self.n3 = (LayerNorm(D, rms=rms) for _ in range(3))
        self.attn = HeadChunkedAttention(D, H, Hkv, U, keep=None)
        self.mlp, self.ce = TiledSwiGLU(D, F, 256), TiledCrossEntropy(D, V, 256)

    def masks(self, p, step):
        return [upipe.Dropout(p, seed=1234, call=3 * step + i) for i in range(3)]

    def forward(self, tokens, labels, p=0.1, step=0, recompute=False):
        d = self.masks(p, step)
        x = dropout(self.emb(tokens), d[0])

        def block(x):
            y, s = self.n2(self.attn(self.n1(x)), x, d[1])
            return self.n3(self.mlp(y), s, d[2])[0]

        y = checkpoint(block, x, use_reentrant=False) if recompute else block(x)
        return self.ce(y, labels)


@pytest.mark.parametrize("rms", [True, False])
def test_a_model_has_gradients_everywhere_and_by_recomputation(rms):
    """Gradients of every parameter; the same bits when the block is computed
    again in the backward; other masks in another step."""
    torch.manual_seed(5)
    m = _Model(rms=rms)
    tokens, labels = _tokens(70, 300, 512), _tokens(71, 300, 512).int()
    grads = []
    for kw in (dict(), dict(recompute=True), dict(step=1)):
        m.zero_grad()
        m(tokens, labels, **kw).backward()
        for n, p in m.named_parameters():
            assert p.grad is not None and torch.isfinite(p.grad).all() and p.grad.abs().max() > 0, n
        grads.append([p.grad.clone() for p in m.parameters()])
    assert all(torch.equal(a, b) for a, b in zip(grads[0], grads[1]))
    assert not all(torch.equal(a, b) for a, b in zip(grads[0], grads[2]))
    status_ok()


def test_gradients_of_a_model_by_differences():
    """The loss along a direction of the norms' weights and of the table, against
    the gradients.  Without masks; the step is large enough that the loss's own
    fp32 and the stages' bf16 rounding (2^-8 of numbers around one, averaged over
    L D elements, so some 1e-5 of the loss) stay below a tenth of the difference."""
    torch.manual_seed(6)
    m = _Model(rms=False)
    tokens, labels = _tokens(72, 300, 512), _tokens(73, 300, 512).int()
    m(tokens, labels, p=0.0).backward()
    for p in (m.n1.w, m.n3.w, m.n3.b, m.emb.w):
        g = p.grad.clone()
        v = g / g.norm()
        h = 0.2
        with torch.no_grad():
            p += h * v
            up = float(m(tokens, labels, p=0.0))
            p -= 2 * h * v
            down = float(m(tokens, labels, p=0.0))
            p += h * v
        want = float((g * v).sum())
        assert abs((up - down) / (2 * h) - want) <= 0.1 * want + 1e-4, (up, down, want)


def test_calls_from_fresh_threads_give_the_same_bits():
    L, D, V = 3000, 520, 700
    t, dy, x = _tokens(80, L, V), _randn(81, L, D), _randn(82, L, D)
    w, d = torch.ones(D, device="cuda"), upipe.Dropout(0.1, seed=2)
    calls = [lambda: upipe.embed_backward(t, dy, V), lambda: upipe.layer_norm_backward(x, w, dy, dy, dropout=d),
             lambda: upipe.layer_norm_forward(x, w, w, residual=dy), lambda: upipe.dropout_forward(d, x, dy),
             lambda: upipe.layer_norm_backward(x[:, :256].contiguous(), w[:256], dy[:, :256].contiguous()),
             lambda: upipe.embed_backward(t[:500].contiguous(), dy[:500], V)]
    want = [f() for f in calls]
    torch.cuda.synchronize()
    got = [None] * len(calls)

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                out = calls[i]()
            torch.cuda.current_stream().synchronize()
            got[i] = out

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    for a, b in zip(got, want):
        for u, v in zip(a if isinstance(a, tuple) else (a,), b if isinstance(b, tuple) else (b,)):
            assert torch.equal(u, v)
    status_ok()


@pytest.mark.parametrize("L", [260, 9000])
def test_captured_training_step_draws_a_new_mask_per_replay(L):
    """Embedding, dropout, norms and their gradients through autograd, captured
    after a warm-up on a side stream, replayed on new tokens with the step
    counter moved on: each replay is the eager step of its number."""
    V, D = 300, 264
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    emb, n1, n2 = TokenEmbedding(V, D), LayerNorm(D, rms=True), LayerNorm(D)
    tokens, dy, dz = _tokens(90, L, V), _randn(91, L, D), _randn(92, L, D)
    masks = [upipe.Dropout(0.3, seed=6, call=1000 * i, step=step) for i in range(2)]

    def run():
        x = dropout(emb(tokens), masks[0])
        y, s = n2(n1(x), x, masks[1])
        return (y, s, *torch.autograd.grad((y, s), (emb.w, n1.w, n2.w, n2.b), (dy, dz)))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    seen = []
    for i in range(3):
        step.fill_(i)
        tokens.copy_(_tokens(93 + i // 2, L, V))
        graph.replay()
        torch.cuda.synchronize()
        want = run()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        seen.append(got[0].clone())
    assert not torch.equal(seen[0], seen[1])  # the same tokens, another mask
    # the counter holds a Dropout's call apart: step 2 is call + 2
    x = _randn(95, L, D)
    assert torch.equal(dropout(x, masks[1]), dropout(x, upipe.Dropout(0.3, seed=6, call=1002)))
    status_ok()


def test_a_tied_tables_gradient_is_added_to_the_heads():
    """Head and embedding share a table: the head's gradient is written, the
    embedding's added to it."""
    L, V, D = 400, 512, 256
    table = _randn(100, V, D, std=0.05).float()
    tokens, labels = _tokens(101, L, V), _tokens(102, L, V).int()
    h = upipe.embed_forward(tokens, table)
    _, dh, dW = upipe.ce_loss(h, table.bfloat16(), labels, 1.0 / L, 128)
    want = dW + upipe.embed_backward(tokens, dh, V)
    upipe.embed_bwd(tokens, dh, dW, add=True)
    # one rounding of the sum either way, of numbers that differ by the product's: two units of 2^-24
    assert ((dW - want).abs() <= 2.0 ** -22 * want.abs() + 1e-12).all()
    # two batches into one gradient, as one of both
    both = upipe.embed_backward(torch.cat([tokens, tokens]), torch.cat([dh, dh]), V)
    g = upipe.embed_backward(tokens, dh, V)
    upipe.embed_bwd(tokens, dh, g, add=True)
    assert_close(f64(g) * L, f64(both) * L, "two batches", weight_grad=True)
    status_ok()


def test_launches_are_counted_and_profiled_by_kind():
    x, w, t = _randn(110, 64, 256), torch.ones(256, device="cuda"), _tokens(111, 64, 30)
    big = _tokens(112, 9000, 30)
    upipe.profile_read()
    upipe.profile_enable(True)
    try:
        n0 = upipe.launch_count()
        upipe.embed_forward(t, w.expand(30, 256).contiguous())
        upipe.embed_backward(t, x, 30)
        upipe.embed_backward(big, x[:1].expand(9000, 256), 30)
        upipe.dropout_forward(upipe.Dropout(0.5), x)
        upipe.layer_norm_forward(x, w)
        upipe.layer_norm_backward(x, w, x)
        n = upipe.launch_count() - n0
    finally:
        upipe.profile_enable(False)
    kinds = {k: v[1] for k, v in upipe.profile_read().items() if v[1]}
    assert kinds == dict(embed_fwd=1, embed_sort=1 + 2, embed_bwd=4, dropout=1, layer_norm_fwd=1, layer_norm_bwd=1,
                         norm_sum=1)
    assert n == sum(kinds.values())
