"""GPU parity of the norms where a team of warps walks over several rows, and of
masks whose counter passes 32 bits inside the tensor, against the fp64 oracle.

Rows: the bounds of test_gpu_residual.py hold.  Its 1e-5 of a column's terms
covers 167 additions one after another (of 2^-24 each).  A column's sum over L
rows goes through the rows of a team, the teams of a CTA (at most 32), a fixed
tree over at most 152 CTAs (5 one after another, then 2 and 8): at the longest
below, 150000 rows of one warp each on 152 SMs of 32 warps, 31 + 32 + 5 + 2 + 8
= 78.  The rounding of n in each term has its own share there.

Masks: element e of a tensor whose first element is number `first` takes its
word from the block (first + e) / 4, whose upper 32 bits change every 2^34
elements.  Compared bit for bit."""

import numpy as np
import pytest
import torch

from headwise_chunked_context_gb300 import upipe
from oracle import residual_oracle as res
from tests.gpu_common import ensure_lib, status_ok
from tests.test_gpu_residual import _check_norm, _check_norm_bwd, _inside, _near_sum, _randn, _weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


# L, D with three rows or more for some teams, however the rows are laid out (rows_at_once in
# test_residual_case_sizes.py): one vector a lane, less than a warp and a whole one; two vectors, one warp and three;
# four vectors, one warp (whole and not) and two; many rows a team
ROWS = [(10000, 64), (10000, 256), (9800, 264), (9800, 512), (4900, 1032), (4900, 1536), (9800, 1024), (9800, 1000),
        (4900, 2048), (4900, 1800), (150000, 64), (40000, 264)]


@pytest.mark.parametrize("L,D", ROWS)
@pytest.mark.parametrize("rms,bias,given,p", [(False, True, False, None), (True, False, True, None),
                                              (True, False, True, 0.2), (False, True, True, 0.2),
                                              (False, False, False, 0.5)])
def test_norms_of_several_rows_a_team_match_oracle(L, D, rms, bias, given, p):
    x, r, (w, b) = _randn(1, L, D, std=2.0, mean=0.5), _randn(2, L, D, std=3.0) if given else None, _weights(D, D)
    b = b if bias else None
    mask = dict(p=p, seed=77, call=L, first=16) if p is not None else {}
    d = upipe.Dropout(**mask) if mask else None
    y, s = upipe.layer_norm_forward(x, w, b, eps=1e-5, rms=rms, residual=r, dropout=d)
    if given or mask:
        _near_sum(s, x, r, mask, "s")
    _check_norm(y, s, w, b, 1e-5, rms, "y")
    del x, r
    dy, ds = _randn(3, L, D), _randn(4, L, D) if given else None
    got = upipe.layer_norm_backward(s, w, dy, ds, eps=1e-5, rms=rms, bias=bias, dropout=d)
    _check_norm_bwd(got, s, w, dy, ds, 1e-5, rms, mask)
    status_ok()


TURN = 1 << 34  # elements between two values of the upper word

# L, D, and how many vectors of 8 elements stand before the change: at the tensor's ends, inside one thread's vectors of
# a dense tensor (256 apart) and of a row, between rows, in a row that a team comes to later
CROSSINGS = [(6, 4096, 1), (6, 4096, 300), (6, 4096, 1724), (6, 4096, 3071), (77, 1032, 40 * 129), (77, 1032, 5000),
             (2, 16384, 2050), (10000, 64, 40000), (10000, 64, 40003), (9800, 264, 300000), (4900, 2048, 1200001)]


@pytest.mark.parametrize("L,D,before", CROSSINGS)
@pytest.mark.parametrize("turns", [1, 5])
def test_masks_whose_counter_passes_32_bits_are_the_oracles(L, D, before, turns):
    mask = dict(p=0.4, seed=0x9876543210, call=(3 << 32) + 7, first=turns * TURN - 8 * before)
    d = upipe.Dropout(**mask)
    keep = torch.from_numpy(res.keep(L, D, **mask)).cuda()
    one, zero = torch.ones(L, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(L, D, dtype=torch.bfloat16, device="cuda")
    (_, wide), (_, base), (_, out) = _inside(one), _inside(zero), _inside(zero)
    assert torch.equal(upipe.dropout_forward(d, one) != 0, keep)
    assert torch.equal(upipe.dropout_forward(d, one, zero) != 0, keep)
    for r in (None, base):
        upipe.dropout_apply(d, wide, r, out)
        assert torch.equal(out != 0, keep)
    w = torch.ones(D, device="cuda")
    dy = _randn(5, L, D)
    for rms in (False, True):
        b = None if rms else w
        for r in (None, zero):
            assert torch.equal(upipe.layer_norm_forward(one, w, b, rms=rms, residual=r, dropout=d)[1] != 0, keep)
        for ds in (None, one):
            dx, dres, _, _ = upipe.layer_norm_backward(dy, w, dy + one, ds, rms=rms, bias=not rms, dropout=d)
            assert torch.equal(dx != 0, keep & (dres != 0)) and float((dres != 0).float().mean()) > 0.9
    status_ok()
