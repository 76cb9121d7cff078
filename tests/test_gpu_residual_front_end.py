"""Embedding, dropout and norms through the autograd front end on tensors that
stand and change as a training program's do."""

import pytest
import torch
from torch.utils.checkpoint import checkpoint

from headwise_chunked_context_gb300 import upipe
from headwise_chunked_context_gb300.modules import LayerNorm, TokenEmbedding, dropout
from tests.gpu_common import ensure_lib, status_ok

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def _randn(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").bfloat16()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("at", [1, 2, 3])
def test_a_table_inside_a_flat_buffer_reads_as_one_of_its_own(dtype, at):
    V, D = 40, 264
    w, dy = _randn(0, V, D).to(dtype), _randn(1, 50, D)
    tokens = torch.arange(50, device="cuda") % 37 - 1
    flat = torch.empty(V * D + 4, dtype=dtype, device="cuda")
    emb = TokenEmbedding(V, D, scale=3.0)
    emb.w = torch.nn.Parameter(flat[at:at + V * D].view(V, D).copy_(w))
    assert emb.w.data_ptr() % 16
    y = emb(tokens)
    y.backward(dy)
    assert torch.equal(y, upipe.embed_forward(tokens, w, 3.0))
    assert emb.w.grad.dtype == dtype and torch.equal(emb.w.grad, upipe.embed_backward(tokens, dy, V, 3.0).to(dtype))
    status_ok()


@pytest.mark.parametrize("recompute", [False, True])
def test_a_step_moved_before_the_backward_is_noticed_with_recomputation_too(recompute):
    L, D = 70, 264
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    d, m, x = upipe.Dropout(0.3, seed=1, call=4, step=step), LayerNorm(D), _randn(2, L, D).requires_grad_()
    for block in (lambda x: dropout(x, d, x), lambda x: m(x, x, d)[0], lambda x: m(x, None, d)[1]):
        def run(recompute=recompute):
            return checkpoint(block, x, use_reentrant=False) if recompute else block(x)

        want = torch.autograd.grad(run(False).float().square().sum(), x)[0]
        assert torch.equal(torch.autograd.grad(run().float().square().sum(), x)[0], want)
        step += 1
        y = run()
        step += 1
        with pytest.raises(RuntimeError, match="modified by an inplace operation|step .* has changed"):
            y.float().square().sum().backward()
        step -= 2
    status_ok()


def test_a_step_whose_memory_is_replaced_is_read_where_it_is():
    x = _randn(3, 40, 520)
    step = torch.tensor([5], device="cuda")
    d = upipe.Dropout(0.4, seed=8, call=100, step=step)
    for n in (5, 9):
        step.data = torch.tensor([n], device="cuda")  # another tensor's memory; the old one's is free
        assert torch.equal(upipe.dropout_forward(d, x), upipe.dropout_forward(upipe.Dropout(0.4, seed=8, call=100 + n), x))
    status_ok()
