"""The sizes of the GPU tests of norms and masks do what those tests say of
them (CPU)."""

import os
import re

import numpy as np
import pytest

from oracle import residual_oracle as res
from tests.test_gpu_residual_rows import CROSSINGS, ROWS, TURN

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "headwise_chunked_context_gb300",
                    "csrc")


def rows_at_once(D):
    """The most rows that the norm kernels can hold at once: a warp holds at most
    four vectors of 8 a lane, an SM kMostWarps warps, and there are 152."""
    code = open(os.path.join(CSRC, "residual.cu")).read()
    warps = int(re.search(r"constexpr int kMostWarps = (\d+);", code).group(1))
    return 152 * (warps // -(-D // 1024))


@pytest.mark.parametrize("L,D", ROWS)
def test_some_team_walks_over_three_rows(L, D):
    assert L > 2 * rows_at_once(D)


def test_some_teams_walk_over_tens_of_rows():
    assert max(L // rows_at_once(D) for L, D in ROWS) >= 30


@pytest.mark.parametrize("L,D,before", CROSSINGS)
def test_the_counters_upper_word_changes_inside_the_tensor(L, D, before):
    """... and a mask whose upper word stays what it was at the first element is
    another one."""
    assert 0 < 8 * before < L * D
    rows = slice(max(0, 8 * before // D - 1), 8 * before // D + 2)
    L, skipped = len(range(*rows.indices(L))), rows.start * D
    first = 5 * TURN - 8 * before + skipped
    e = np.uint64(first) + np.arange(L * D, dtype=np.uint64)
    block, low = e >> np.uint64(2), np.uint64(0xFFFFFFFF)
    words = res.philox([block & low, np.full_like(block, (first >> 2) >> 32), np.full_like(e, 7), np.full_like(e, 3)],
                       (0x76543210, 0x98))
    stale = (np.choose((e & np.uint64(3)).astype(np.int64), words) >= np.uint64(res.steps_of(0.4))).reshape(L, D)
    keep = res.keep(L, D, 0.4, seed=0x9876543210, call=(3 << 32) + 7, first=first)
    at = 8 * before - skipped
    assert np.array_equal(keep.ravel()[:at], stale.ravel()[:at])
    assert not np.array_equal(keep.ravel()[at:], stale.ravel()[at:])
