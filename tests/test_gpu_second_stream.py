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
