"""How exactly the norm's gradient adds up its weight gradient (MI355X).

dweight = sum over rows of dy xh goes through, u = 2^-24 each:
  a workgroup's rows, one FMA each: ceil(rows / (grid per)), the grid being one workgroup per CU (256), or two
  from 4096 rows on, and `per` rows at once (4 waves: 4, 2 or 1);
  its partial sums: each of a column's 64 lanes adds every 64th, ceil(partials / 64);
  a tree over the 64: 6.
"""
import pytest

import block_scaled_precision_fp8_amd as bs
from gpu_common import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def additions(rows, k):
    pieces = -(-k // 512)
    group = pieces if pieces <= 16 else -(-pieces // (2 if pieces <= 32 else 4))
    per = 1 if group >= 4 else 4 // group
    need, most = -(-rows // per), 512 if rows >= 4096 else 256
    grid = -(-need // -(-need // most))
    return -(-rows // (grid * per)) + -(-grid * per // 64) + 6


@pytest.mark.parametrize("rows,k", [(64, 2048), (256, 5001), (777, 5001), (1025, 4100), (3000, 600), (6000, 130), (64, 20001)])
def test_weight_gradient_of_a_large_row_among_small_ones(rows, k):
    """One row of 2^24 among ones: an addition of 1 to the large sum loses it, so the error counts the additions
    that the large sum went through."""
    import torch
    say(f"rmsnorm_backward {rows}x{k}: 2^24 among ones")
    h, rstd = torch.ones((rows, k), device="cuda"), torch.ones(rows, device="cuda")
    want = 2.0 ** 24 + rows - 1
    for row in (0, rows // 3, rows - 1):
        dy = torch.ones((rows, k), device="cuda")
        dy[row] = 2.0 ** 24
        for start in (None, torch.full((k,), 3.0, device="cuda")):
            _, dw = bs.rmsnorm_backward(dy, h, rstd, dweight=None if start is None else start.clone(), accumulate=start is not None)
            exact, n = (want, additions(rows, k)) if start is None else (want + 3, additions(rows, k) + 1)
            off = float((dw.double() - exact).abs().max())
            say(f"row {row}: off by {off}, {n} additions")
            assert off <= n * U * exact, f"{off} of {n * U * exact}"
