"""The autograd front end and the binding of embedding, dropout and norms, as
far as the host goes (CPU): what they hand to the library, which is stood in
for where a call would reach it."""

import pytest
import torch
from torch.utils.checkpoint import checkpoint

from headwise_chunked_context_gb300 import modules, upipe


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float64])
@pytest.mark.parametrize("place", ["aligned", "off", "strided"])
def test_tables_reach_the_lookup_dense_on_a_16_byte_boundary(monkeypatch, dtype, place):
    """A table may be a parameter inside a flat buffer, which starts at any element."""
    V, D = 30, 264
    w = torch.randn(V, D, generator=torch.Generator().manual_seed(0)).to(dtype)
    if place == "off":
        flat = torch.empty(V * D + 4, dtype=dtype)
        at = next(i for i in range(4) if (flat.data_ptr() + i * flat.element_size()) % 16)
        w = flat[at:at + V * D].view(V, D).copy_(w)
    elif place == "strided":
        w = w.t().contiguous().t()
    emb = modules.TokenEmbedding(V, D, device="cpu")
    emb.w = torch.nn.Parameter(w)
    seen = []

    def lookup(tokens, W, scale):
        seen.append(W)
        return W[tokens].to(torch.bfloat16)

    monkeypatch.setattr(upipe, "embed_forward", lookup)
    monkeypatch.setattr(upipe, "embed_backward",
                        lambda tokens, dy, V, scale: torch.zeros(V, dy.shape[1]).index_add_(0, tokens, dy.float()))
    tokens = torch.tensor([3, 3, 0, 29])
    emb(tokens).float().sum().backward()
    (W,) = seen
    assert W.data_ptr() % 16 == 0 and W.is_contiguous()
    assert W.dtype == (torch.bfloat16 if dtype == torch.bfloat16 else torch.float32)
    assert torch.equal(W, w.to(W.dtype))
    if place == "aligned" and dtype != torch.float64:
        assert W.data_ptr() == w.data_ptr()  # read as it is
    want = torch.zeros(V, D, dtype=dtype)
    want[3], want[0], want[29] = 2, 1, 1
    assert emb.w.grad.dtype == dtype and torch.equal(emb.w.grad, want)


class _Mask:
    """Stands in for upipe.Dropout: x (1 + step), so that each step is another mask."""

    def __init__(self, step):
        self.step = step


@pytest.fixture
def plain(monkeypatch):
    """The calls that dropout and LayerNorm make, of a stand-in's step alone."""
    def factor(drop):
        return 1 if drop is None or drop.step is None else 1 + drop.step.to(torch.bfloat16)

    def norm(x, w, b, eps, rms, residual, drop):
        s = x * factor(drop)
        return s * w.bfloat16(), s

    def norm_back(s, w, dy, ds, eps, rms, bias, drop):
        d = dy * w.bfloat16() if ds is None else dy * w.bfloat16() + ds
        return d * factor(drop), d, (dy * s).float().sum(0), dy.float().sum(0)

    monkeypatch.setattr(upipe, "dropout_forward", lambda drop, x, r=None: x * factor(drop))
    monkeypatch.setattr(upipe, "dropout_backward", lambda drop, dy: dy * factor(drop))
    monkeypatch.setattr(upipe, "layer_norm_forward", norm)
    monkeypatch.setattr(upipe, "layer_norm_backward", norm_back)
    return modules.LayerNorm(8, device="cpu")


@pytest.mark.parametrize("kind", ["dropout", "norm", "sum alone"])
def test_a_step_moved_before_a_recomputation_is_noticed(plain, kind):
    """Under activation checkpointing the step that a backward finds saved is the
    recomputation's: the mask drawn again would be another one, without an error."""
    step = torch.ones(1, dtype=torch.int64)
    d, x = _Mask(step), torch.ones(4, 8, dtype=torch.bfloat16, requires_grad=True)

    def block(x):
        if kind == "dropout":
            return modules.dropout(x, d)
        y, s = plain(x, x, d)
        return s * 2 if kind == "sum alone" else y

    for recompute in (False, True):
        def run():
            return checkpoint(block, x, use_reentrant=False) if recompute else block(x)

        run().float().sum().backward()  # as it was
        step += 1
        run().float().sum().backward()  # moved between steps
        y = run()
        step += 1
        with pytest.raises(RuntimeError, match="modified by an inplace operation|step .* has changed"):
            y.float().sum().backward()


def test_steps_of_inference_mode_run_where_no_backward_follows(plain):
    with torch.inference_mode():
        d = _Mask(torch.ones(1, dtype=torch.int64))
    x = torch.ones(4, 8, dtype=torch.bfloat16)
    with torch.no_grad():
        assert torch.equal(modules.dropout(x, d), 2 * x)
        assert torch.equal(plain(x, None, d)[1], 2 * x)


class _Counter:
    """A CUDA tensor of one int64 element, as far as a mask's description reads it."""
    is_cuda, dtype, shape, device = True, torch.int64, (1,), "cuda:0"

    def __init__(self):
        self.at, self.n, self.index = 1 << 20, 1, 0

    def numel(self):
        return self.n

    def data_ptr(self):
        return self.at

    def get_device(self):
        return self.index


def test_a_masks_step_is_looked_up_by_each_call():
    """A counter's memory may be replaced (``step.data = ...``, a module moved): the
    kernels read where it is, not where it was."""
    step = _Counter()
    d = upipe.Dropout(0.25, seed=(1 << 64) - 1, call=3, first=64, step=step)
    for step.at in (1 << 20, 1 << 24):
        c = upipe._drop(d, 0)._obj
        assert (c.p, c.seed, c.call, c.first, c.step) == (0.25, (1 << 64) - 1, 3, 64, step.at)
    step.n = 0  # its memory is gone
    with pytest.raises(ValueError, match="step"):
        upipe._drop(d, 0)
    step.n, step.index = 1, 1
    with pytest.raises(ValueError, match="step is on"):
        upipe._drop(d, 0)
    assert upipe._drop(upipe.Dropout(0.25, first=8), 0)._obj.step is None


@pytest.mark.parametrize("name", ["seed", "call", "first"])
def test_a_masks_numbers_are_whole(name):
    """A part of a number would be cut off: two masks that are told apart by it
    would be one."""
    for bad in (0.5, 1.5, 8.25, -0.5, float("nan"), float("inf")):
        with pytest.raises(ValueError, match=name):
            upipe.Dropout(0.1, **{name: bad})
    for good in (8, 8.0, torch.tensor(8).numpy()[()]):
        d = upipe.Dropout(0.1, **{name: good})
        assert getattr(d, name) == 8 and type(getattr(d, name)) is int
    assert getattr(upipe.Dropout(0.1, **{name: 2.0 ** 62}), name) == 1 << 62
