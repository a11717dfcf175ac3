"""Grouped products without K values, at sizes where their tiles pass what one launch counts (MI355X)."""
import pytest

import block_scaled_precision_fp8_amd as bs
from gpu_common import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("groups,N,at", [(1000, 1 << 21, 998), (1, (1 << 30) + 72, 0)])
def test_more_tiles_than_a_launch_counts(groups, N, at):
    """One row, of group `at`: 16-column tiles of 64 threads, more than 2^32 threads in all.  Every element is
    beta C, or zero, and the row before is left as it was."""
    import torch
    say(f"grouped, K = 0, {groups} groups, N {N}")
    assert (N + 15) // 16 * groups * 64 >= 1 << 32
    u8 = dict(dtype=torch.uint8, device="cuda")
    a, sa, b, sb = torch.zeros((2, 0), **u8), torch.zeros((0, 2, 4), **u8), torch.zeros((groups, N, 0), **u8), \
        torch.zeros((groups, 0, (N + 127) // 128, 4), **u8)
    o = torch.ones(groups + 1, dtype=torch.int32, device="cuda")
    o[at + 1:] = 2
    d = torch.full((2, N), 3.0, dtype=torch.bfloat16, device="cuda")
    bs.scaled_gemm_grouped_block128(a, sa, b, sb, o, c=d, beta=0.5, d=d)
    # (truth values, not tensors: a failure would print those element by element)
    kept, scaled = bool((d[0] == 3.0).all()), bool((d[1] == 1.5).all())
    assert kept and scaled
    bs.scaled_gemm_grouped_block128(a, sa, b, sb, o, d=d)
    kept, zeros = bool((d[0] == 3.0).all()), not bool(d[1].any())
    assert kept and zeros
