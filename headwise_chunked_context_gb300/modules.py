"""PyTorch autograd front end of the library: the head-chunked attention
layer, the sequence-tiled SwiGLU MLP and the tiled LM-head loss as
``torch.autograd.Function`` s and ``nn.Module`` s, so that a training loop
can use them in place of its own attention, MLP and loss; and, for a layer
with projections of its own, what stands between them: rotary positions, the
norms of queries and keys, and attention with a sliding window and sinks.

Every forward and backward runs the library's kernels through the binding
(``upipe.py``); nothing here computes.  Weights are held as fp32 master
parameters: each call hands their bf16 rounding to the kernels and returns
the kernels' fp32 weight gradients, so no precision is lost in the gradient
sums.  Activations are bf16 CUDA tensors.

Before a backward is captured into a CUDA graph, drop the eager graphs of the
same leaves: PyTorch accumulates a leaf's gradient on the stream of its first
use for as long as such a graph lives, and a capture cannot wait for that stream.
"""

from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from headwise_chunked_context_gb300 import upipe


# ------------------------------------------------------------------ attention

class _AttentionFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, wqkv, wo, cfg, keep):
        wqkv_b, wo_b = wqkv.to(torch.bfloat16), wo.to(torch.bfloat16)
        out, lse, kept = upipe.layer_forward(cfg, x.contiguous(), wqkv_b, wo_b, keep_o=keep)
        ctx.save_for_backward(x, wqkv_b, wo_b, lse)
        ctx.kept, ctx.cfg = kept, cfg
        return out

    @staticmethod
    def backward(ctx, dout):
        x, wqkv_b, wo_b, lse = ctx.saved_tensors
        dx, dwqkv, dwo = upipe.layer_backward(ctx.cfg, x.contiguous(), wqkv_b, wo_b,
                                              dout.to(torch.bfloat16).contiguous(), lse, ctx.kept)
        ctx.kept = None
        return dx, dwqkv, dwo, None, None


class HeadChunkedAttention(torch.nn.Module):
    """One GQA/RoPE causal attention layer computed U query heads at a time
    (upipe_attn_fwd / upipe_attn_bwd): ``out = Attention(x)`` for x [L, D]
    bf16.  keep: None (the backward recomputes each chunk's Q/K/V and O),
    "device_o" (O kept on the device) or "host" (O kept in page-locked host
    memory, the fastest)."""

    def __init__(self, D: int, H: int, Hkv: int, U: int, rope_theta: float = 500000.0, keep="host",
                 device="cuda", init_std: float = 0.02):
        super().__init__()
        self.D, self.H, self.Hkv, self.U, self.rope_theta = D, H, Hkv, U, rope_theta
        if keep not in (None, "device_o", "host"):
            raise ValueError(f"keep: expected None, 'device_o' or 'host', got {keep!r}")
        self.keep = {None: False, "device_o": True, "host": "host"}[keep]
        self.wqkv = torch.nn.Parameter(torch.randn((H + 2 * Hkv) * 128, D, device=device) * init_std)
        self.wo = torch.nn.Parameter(torch.randn(D, H * 128, device=device) * init_std)

    def forward(self, x):
        cfg = upipe.Config(L=x.shape[0], D=self.D, H=self.H, Hkv=self.Hkv, U=self.U, rope_theta=self.rope_theta)
        return _AttentionFn.apply(x, self.wqkv, self.wo, cfg, self.keep)


# ------------------------------------------------------------------- MLP

class _MlpFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, wgu, wd, T):
        wgu_b, wd_b = wgu.to(torch.bfloat16), wd.to(torch.bfloat16)
        y = upipe.mlp_forward(x.contiguous(), wgu_b, wd_b, T)
        ctx.save_for_backward(x, wgu_b, wd_b)
        ctx.T = T
        return y

    @staticmethod
    def backward(ctx, dy):
        x, wgu_b, wd_b = ctx.saved_tensors
        dx, dwgu, dwd = upipe.mlp_backward(x.contiguous(), wgu_b, wd_b, dy.to(torch.bfloat16).contiguous(), ctx.T)
        return dx, dwgu, dwd, None


class TiledSwiGLU(torch.nn.Module):
    """SwiGLU MLP computed T rows at a time (upipe_mlp_fwd / _bwd):
    ``y = (silu(x Wg^T) * (x Wu^T)) Wd^T`` for x [L, D] bf16; Wgu = [Wg; Wu]."""

    def __init__(self, D: int, F: int, T: int = 8192, device="cuda", init_std: float = 0.02):
        super().__init__()
        self.T = T
        self.wgu = torch.nn.Parameter(torch.randn(2 * F, D, device=device) * init_std)
        self.wd = torch.nn.Parameter(torch.randn(D, F, device=device) * init_std)

    def forward(self, x):
        return _MlpFn.apply(x, self.wgu, self.wd, self.T)


# ------------------------------------------------------------------- loss

class _CeFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, w, labels, T):
        valid = int((labels >= 0).sum())
        scale = 1.0 / max(1, valid)
        # loss and both gradients in one pass over the vocabulary, tile by tile
        loss, dh, dw = upipe.ce_loss(h.contiguous(), w.to(torch.bfloat16), labels.to(torch.int32).contiguous(),
                                     scale, T)
        ctx.save_for_backward(dh, dw)
        return loss.sum() * scale

    @staticmethod
    def backward(ctx, g):
        dh, dw = ctx.saved_tensors
        return (dh * g).to(torch.bfloat16), dw * g, None, None


class TiledCrossEntropy(torch.nn.Module):
    """Mean next-token cross-entropy of the LM head computed T rows at a time
    (upipe_ce_fwd_bwd): ``loss = mean_i logsumexp(h_i W^T) - (h_i W^T)[y_i]``
    over labels >= 0.  The gradients are formed together with the loss."""

    def __init__(self, D: int, V: int, T: int = 4096, device="cuda", init_std: float = 0.02):
        super().__init__()
        self.T = T
        self.w = torch.nn.Parameter(torch.randn(V, D, device=device) * init_std)

    def forward(self, h, labels):
        return _CeFn.apply(h, self.w, labels, self.T)


# ------------------- rotary positions, query/key norms, windowed attention

def _heads(t):
    """t in bf16, copied where its heads do not start on 16-byte boundaries or
    its rows are one (a broadcast)."""
    t = t.to(torch.bfloat16)
    *outer, one = t.stride()
    fits = one == 1 and t.data_ptr() % 16 == 0 and all(n == 1 or s > 0 and s % 8 == 0 for n, s in zip(t.shape, outer))
    return t if fits else t.clone(memory_format=torch.contiguous_format)


def _dense(t):
    """t in bf16, copied where it is not dense from a 16-byte boundary on."""
    t = t.to(torch.bfloat16)
    return t if t.is_contiguous() and t.data_ptr() % 16 == 0 else t.clone(memory_format=torch.contiguous_format)


class _RopeFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, rope, pos0, positions):
        ctx.save_for_backward(positions)  # which also sees to it that they are the forward's
        ctx.rope, ctx.pos0 = rope, pos0
        return upipe.rope_forward(rope, _heads(q), _heads(k), pos0, positions)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk):
        dq, dk = upipe.rope_backward(ctx.rope, _heads(dq), _heads(dk), ctx.pos0, *ctx.saved_tensors)
        return dq, dk, None, None, None


def rotate(q, k, rope, pos0: int = 0, positions=None):
    """q [L, H, d] and k [L, Hkv, d] rotated by `rope` (upipe.Rope) to the
    positions pos0, pos0 + 1, ... or `positions` [L] int32, differentiable."""
    return _RopeFn.apply(q, k, rope, pos0, positions)


class _QKNormRopeFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, wq, wk, rope, eps, pos0, positions):
        q, k, wq, wk = _heads(q), _heads(k), wq.float(), wk.float()
        ctx.save_for_backward(q, k, wq, wk, positions)
        ctx.args = rope, eps, pos0
        return upipe.qk_norm_rope_forward(rope, q, k, wq, wk, eps, pos0, positions)

    @staticmethod
    @once_differentiable
    def backward(ctx, dqo, dko):
        q, k, wq, wk, positions = ctx.saved_tensors
        rope, eps, pos0 = ctx.args
        dq, dk, dwq, dwk = upipe.qk_norm_rope_backward(rope, q, k, wq, wk, _heads(dqo), _heads(dko), eps, pos0,
                                                       positions)
        return dq, dk, dwq, dwk, None, None, None, None


class QKNormRope(torch.nn.Module):
    """RMS norm of each query and key head (weights wq, wk [d] fp32) and the
    rotation by `rope` in one pass: (q [L, H, d], k [L, Hkv, d]) bf16 ->
    (q, k)."""

    def __init__(self, rope, eps: float = 1e-6, device="cuda"):
        super().__init__()
        self.rope, self.eps = rope, eps
        self.wq = torch.nn.Parameter(torch.ones(rope.d, device=device))
        self.wk = torch.nn.Parameter(torch.ones(rope.d, device=device))

    def forward(self, q, k, pos0: int = 0, positions=None):
        return _QKNormRopeFn.apply(q, k, self.wq, self.wk, self.rope, self.eps, pos0, positions)


class _WindowFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, window, sinks):
        q, k, v = _dense(q), _dense(k), _dense(v)
        ctx.cfg = upipe.WindowConfig(L=q.shape[0], H=q.shape[1], Hkv=k.shape[1], window=window, sinks=sinks)
        o, lse = upipe.window_forward(ctx.cfg, q, k, v)
        ctx.save_for_backward(q, k, v, o, lse)
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, do):
        dq, dk, dv = upipe.window_backward(ctx.cfg, *ctx.saved_tensors, _dense(do))
        return dq, dk, dv, None, None


def window_attention(q, k, v, window: int, sinks: int = 0):
    """Causal attention in which query i sees key j iff j <= i and (i - j <
    window or j < sinks): q [L, H, 128], k, v [L, Hkv, 128] -> [L, H, 128],
    bf16, differentiable."""
    return _WindowFn.apply(q, k, v, window, sinks)


__all__ = ["HeadChunkedAttention", "TiledSwiGLU", "TiledCrossEntropy", "QKNormRope", "rotate", "window_attention"]
