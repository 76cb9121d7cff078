"""Workspaces that the binding makes for a call on a given stream come from
that stream's memory: a block of the current stream's, freed a moment ago, may
still be in use by what the current stream has queued."""

import contextlib
import inspect
import re

import pytest
import torch

from headwise_chunked_context_gb300 import synth, upipe
from tests.gpu_common import dev, ensure_lib, status_ok


@pytest.mark.parametrize("given", [None, "a stream"])
def test_workspace_is_allocated_on_the_stream_of_the_call(monkeypatch, given):
    """CPU: which stream is current when the memory is taken."""
    current, taken = [None], []

    @contextlib.contextmanager
    def stream(s):
        current.append(s)
        yield
        current.pop()

    empty = torch.empty

    def recorded(*a, **kw):
        taken.append(current[-1])
        return empty(*a, **kw)

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch, "empty", recorded)
    ws, nbytes = upipe._call_ws(640, None, "cpu", given)
    assert taken == [given] and nbytes == ws.numel() >= 640 and current == [None]


def test_every_call_with_a_workspace_and_a_stream_hands_the_stream_on():
    calls = [f for _, f in inspect.getmembers(upipe, inspect.isfunction)
             if {"ws", "stream"} <= set(inspect.signature(f).parameters) and not f.__name__.startswith("_")]
    assert len(calls) >= 10
    for f in calls:
        text = inspect.getsource(f)
        made = re.findall(r"_ws\((?:[^()]|\([^()]*\))*\)", text.replace("_expect_ws", ""))
        made = [m for m in made if "device" in m]
        assert made and all(m.endswith(".device, stream)") for m in made), f.__name__
        assert "torch.empty" not in text, f.__name__


@pytest.mark.gpu
def test_a_call_on_another_stream_keeps_clear_of_pending_work():
    """A block of the size of the workspaces, freed with many writes to it
    still queued on the current stream, is not where a call on another stream
    puts its workspace: the results have the bits of an ordinary call."""
    ensure_lib()
    L, H, Hkv = 700, 4, 2
    q, k, v, do = dev(*synth.core_inputs(L, H, Hkv))
    w, rope = torch.linspace(0.5, 1.5, 128, device="cuda"), upipe.Rope(128)
    wcfg, ccfg = upipe.WindowConfig(L=L, H=H, Hkv=Hkv, window=90, sinks=3), upipe.Config(L=L, H=H, Hkv=Hkv, U=H)
    o, lse = upipe.window_forward(wcfg, q, k, v)
    co, clse = upipe.core_forward(ccfg, q, k, v)
    grads = [torch.empty_like(t) for t in (q, k, v)]
    norm = [torch.empty_like(t) for t in (q, k, w, w)]
    x, y = (torch.randn(256, 512, device="cuda").bfloat16() for _ in range(2))
    wgu, wd = torch.randn(1024, 512, device="cuda").bfloat16(), torch.randn(512, 512, device="cuda").bfloat16()
    mlp = [torch.empty_like(y), torch.empty(1024, 512, device="cuda"), torch.empty(512, 512, device="cuda")]
    calls = [
        (upipe.window_workspace_bytes(wcfg), grads,
         lambda **kw: upipe.window_bwd(wcfg, q, k, v, o, lse, do, *grads, **kw)),
        (upipe.qk_norm_rope_workspace_bytes(rope, L, H, Hkv), norm,
         lambda **kw: upipe.qk_norm_rope_bwd(rope, q, k, w, w, do, v, *norm, **kw)),
        (upipe.workspace_bytes(ccfg, 1, True), grads,
         lambda **kw: upipe.attn_core_bwd(ccfg, q, k, v, co, clse, do, *grads, **kw)),
        (upipe.mlp_workspace_bytes(256, 512, 512, 128, 1), mlp,
         lambda **kw: upipe.mlp_bwd(x, wgu, wd, y, *mlp, 128, **kw)),
    ]
    other = torch.cuda.Stream()
    for need, outs, call in calls:
        call()
        torch.cuda.synchronize()
        want = [t.clone() for t in outs]
        for t in outs:
            t.zero_()
        torch.cuda.synchronize()
        block = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
        for i in range(300):
            block.fill_(i % 256)
        del block
        call(stream=other)
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
    status_ok()
