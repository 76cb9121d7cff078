"""The library's second stream is joined back into the caller's whatever
becomes of the launches on either."""

import ctypes

import pytest
import torch

from headwise_chunked_context_gb300 import upipe
from tests.gpu_common import ensure_lib

pytestmark = pytest.mark.gpu

LAUNCH = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p)


@pytest.mark.parametrize("own_error", [0, 1])
def test_the_callers_stream_waits_for_the_side_launch(own_error):
    """upipe::launch_beside with a side launch that waits 100 ms (bounded) and
    an own launch that does nothing, with and without an error."""
    lib = ensure_lib()
    beside = lib["_ZN5upipe13launch_besideEiPF9cudaErrorPvP11CUstream_stEiS5_S1_S3_"]
    beside.restype = ctypes.c_int
    beside.argtypes = [ctypes.c_int, LAUNCH, ctypes.c_int, LAUNCH, ctypes.c_void_p, ctypes.c_void_p]
    side = LAUNCH(lambda job, on: int(lib.upipe_debug_wait_timeout(100_000_000, on) != 0))
    own = LAUNCH(lambda job, on: own_error)
    upipe.debug_wait_timeout(1000)  # loads the kernel
    assert upipe.last_device_status() == upipe.UPIPE_ERR_DEVICE_TIMEOUT
    st = torch.cuda.Stream()
    rc = beside(0, side, 0, own, None, st.cuda_stream)
    after = torch.cuda.Event()
    after.record(st)
    waits = not after.query()
    torch.cuda.synchronize()
    assert upipe.last_device_status() == upipe.UPIPE_ERR_DEVICE_TIMEOUT  # the side launch ran
    assert rc == (upipe.UPIPE_ERR_CUDA if own_error else 0)
    assert waits


def test_backwards_from_several_threads_at_once():
    """Four host threads, each with a stream, inputs and a workspace of its
    own: they share the second stream and its events, and every call has the
    bits of a call alone."""
    import threading

    from headwise_chunked_context_gb300 import synth
    ensure_lib()
    jobs = []
    cases = [(700, 4, 2, 90, 3), (1500, 2, 1, 400, 0), (300, 8, 2, 1, 130), (2000, 2, 2, 50, 300)]
    for i, (L, H, Hkv, W, S) in enumerate(cases):
        q, k, v, do = (t.roll(i, 0).contiguous().to("cuda:0") for t in synth.core_inputs(L, H, Hkv))
        cfg = upipe.WindowConfig(L=L, H=H, Hkv=Hkv, window=W, sinks=S)
        o, lse = upipe.window_forward(cfg, q, k, v)
        jobs.append(((cfg, q, k, v, o, lse, do), upipe.window_backward(cfg, q, k, v, o, lse, do), torch.cuda.Stream()))
    torch.cuda.synchronize()
    results = [[] for _ in jobs]

    def work(i):
        args, want, st = jobs[i]
        for _ in range(25):
            out = [torch.empty_like(t) for t in want]
            upipe.window_bwd(*args, *out, stream=st)
            results[i].append(out)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert upipe.last_device_status() == 0
    for (_, want, _), got in zip(jobs, results):
        assert len(got) == 25 and all(torch.equal(a, b) for out in got for a, b in zip(out, want))
