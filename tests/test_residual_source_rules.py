"""Static rules of the residual stream's kernels (CPU): what they may not do
for lack of a lane, and what passes from one kernel to the next."""

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "headwise_chunked_context_gb300",
                    "csrc")


def _code(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def test_team_barriers_are_reached_by_whole_warps():
    """A warp arrives at a named barrier as one: the lanes that branched off
    before it (lane 0 writes the warp's sum) are brought back first, and the
    barrier is the form that does not require them to be."""
    code = _code("residual.cu")
    uses = [m.start() for m in re.finditer(r'asm volatile\("(?:bar|barrier)\.[a-z.]+ ', code)]
    assert uses
    for at in uses:
        assert code[at:].startswith('asm volatile("barrier.sync ')
        assert code[:at].rstrip().endswith("__syncwarp();")


def test_copies_take_no_cache_policy():
    """Asynchronous copies that some lanes or whole warps leave out carry no L2
    policy: with one, a build of the norm's backward whose copies were left out by
    a comparison stopped with an illegal instruction."""
    for name in ("residual.cu", "embed.cu"):
        code = _code(name)
        assert "cache_hint" not in code and "createpolicy" not in code, name


def test_kernels_made_ready_early_begin_by_waiting():
    """Every kernel launched by launch_next waits for the one before it ahead of
    any access to memory."""
    for name in ("residual.cu", "embed.cu"):
        code = _code(name)
        for kernel in set(re.findall(r"launch_next\((\w+)", code)):
            body = code[code.index(kernel + "(const __grid_constant__"):]
            body = body[body.index("{") + 1:]
            first = [s.strip() for s in body.split(";") if s.strip()]
            lines = [s for s in first[:3] if not s.startswith("__shared__")]
            assert lines[0] == "after_previous()", (kernel, lines)
