"""Static rules of the CUDA sources (CPU): every barrier wait goes through the
bounded helpers of sm103_ptx.cuh, those helpers take a limit, and no kernel
traps or asserts on the device."""

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "headwise_chunked_context_gb300",
                    "csrc")
HELPERS = os.path.join(CSRC, "sm103_ptx.cuh")


def _sources():
    return {f: open(os.path.join(CSRC, f)).read() for f in sorted(os.listdir(CSRC)) if f.endswith((".cu", ".cuh"))}


def test_kernels_wait_only_through_the_helpers():
    for name, text in _sources().items():
        if name == "sm103_ptx.cuh":
            continue
        assert "mbarrier.try_wait" not in text and "mbarrier.test_wait" not in text, name


def test_looping_helpers_are_bounded():
    text = open(HELPERS).read()
    # Every helper that loops on a barrier takes the wait control (abort flag,
    # status word, limit) or, while unwinding, the status word.
    for fn in ("mbar_wait", "mbar_spin", "warp_wait"):
        sig = re.search(r"\b" + fn + r"\(([^)]*)\)\s*\{", text)
        assert sig and "const WaitCtl&" in sig.group(1), fn
    sig = re.search(r"\bmbar_wait_drain\(([^)]*)\)\s*\{", text)
    assert sig and "int* status" in sig.group(1)
    # The loops in those helpers compare a clock against a limit.
    for fn in ("mbar_wait", "mbar_spin", "mbar_wait_drain", "warp_wait"):
        body = text[re.search(r"\b" + fn + r"\(", text).start():]
        body = body[:body.index("\n}\n")]
        assert "sm_cycles()" in body, fn


def test_no_device_trap_or_assert():
    for name, text in _sources().items():
        code = re.sub(r"//[^\n]*", "", text)
        assert "__trap" not in code, name
        assert re.search(r"(?<!static_)\bassert\s*\(", code) is None, name


def test_a_copy_ring_is_drained_before_it_is_filled_anew():
    """Two asynchronous copies of one thread into the same shared-memory slot
    have no order unless the first is waited for.  The backward of the norm
    walks the queries and then the keys over one ring, and the queries' last
    steps (zeros past the end) are still open when its loop ends: between that
    loop and the keys' first copies stands a wait for all of them."""
    text = _sources()["qk_rope.cu"]
    body = text[text.index("void __launch_bounds__(kWarps * 32, 2) qk_norm_rope_bwd_kernel"):]
    body = body[:body.index("\n}\n")]
    assert body.count("Loads pipe(") == 1 and body.index("for (int t = 0; t < 2; ++t)") < body.index("Loads pipe(")
    turns, ends = body.index("while (at.unit < units)"), body.index("__shfl_xor_sync(0xffffffffu, gu[i]")
    assert re.search(r"\n    }\n    pipe\.drain\(\);", body[turns:ends])
    drain = re.search(r"void drain\(\) \{(.*?)\n  \}", text, re.S).group(1)
    assert "cp.async.wait_all;" in drain
