"""The autograd front end and the binding of embedding, dropout and norms, as
far as the host goes (CPU): what they hand to the library, which is stood in
for where a call would reach it."""

import pytest
import torch

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
