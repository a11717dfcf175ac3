"""Products of ones, through every entry point and at sizes that reach every kernel form (MI355X).

Every element of A B^T is K then, exactly, in each output type and whatever the order of the sums.  A matrix
instruction's result that is read before it is there lacks the last products, 32 or 64 of K: a bound on
random operands, relative to sum |a b|, lets that pass where K is large, these do not.
"""
import pytest

import block_scaled_precision_fp8_amd as bs
from gpu_common import say

pytestmark = pytest.mark.gpu

ONE = {"e4m3": 0x38, "e5m2": 0x3C}
#: sums that bf16 holds exactly (at most eight significant bits)
DEPTHS = [32, 64, 96, 160, 256, 512, 544, 1024, 2048, 4096]
SHAPES = [(1, 48), (16, 1000), (64, 512), (200, 136), (600, 520), (1300, 2050)]
EPILOGUES = [(1.0, 0.0), (0.5, 1.0)]


def ones(shape, byte):
    import torch
    return torch.full(shape, byte, dtype=torch.uint8, device="cuda")


def check(call, M, N, K, label):
    """call(out, alpha, c, beta) -> D, against alpha K + beta C."""
    import torch
    for out, dt in (("f32", torch.float32), ("bf16", torch.bfloat16), ("f16", torch.float16)):
        for alpha, beta in EPILOGUES:
            c = None if beta == 0.0 else torch.full((M, N), -16.0, dtype=dt, device="cuda")
            d = call(out, alpha, c, beta)
            want = alpha * K + (0.0 if c is None else beta * -16.0)
            wrong = int((d.double() != want).sum())
            assert wrong == 0, f"{label} {out} alpha {alpha} beta {beta}: {wrong} of {d.numel()} elements are not {want}"


@pytest.mark.parametrize("M,N", SHAPES)
@pytest.mark.parametrize("gran", ["tile", "row", "tensor"])
@pytest.mark.parametrize("af,bf", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e5m2", "e5m2")])
def test_fp8(af, bf, gran, M, N):
    import torch
    for K in DEPTHS:
        say(f"ones: fp8 {af} {bf} {gran} {M} x {N} x {K}")
        a, b = ones((M, K), ONE[af]), ones((N, K), ONE[bf])
        count = {"tile": lambda r: (r + 127) // 128 * (K // 32), "row": lambda r: r, "tensor": lambda r: 1}[gran]
        sa, sb = (torch.ones(count(r), device="cuda") for r in (M, N))
        check(lambda out, alpha, c, beta: bs.scaled_gemm_granular(a, sa, b, sb, af, bf, gran, gran, out, alpha, c, beta),
              M, N, K, f"{af} {bf} {gran} {M} x {N} x {K}")


@pytest.mark.parametrize("M,N", SHAPES)
@pytest.mark.parametrize("block,scale", [(32, "e8m0"), (16, "e8m0"), (8, "e8m0"), (16, "f16"), (32, "bf16"), (8, "f16")])
def test_mx(block, scale, M, N):
    import torch
    for K in DEPTHS:
        say(f"ones: mx {block} {scale} {M} x {N} x {K}")
        a, b = ones((M, K // 2), 0x22), ones((N, K // 2), 0x22)
        if scale == "e8m0":
            sa, sb = (ones((r, K // block), 127) for r in (M, N))
        else:
            dt = {"f16": torch.float16, "bf16": torch.bfloat16}[scale]
            sa, sb = (torch.ones((r, K // block), dtype=dt, device="cuda") for r in (M, N))
        check(lambda out, alpha, c, beta: bs.scaled_gemm_mx(a, sa, b, sb, block, scale, out, alpha, c, beta),
              M, N, K, f"mx {block} {scale} {M} x {N} x {K}")


@pytest.mark.parametrize("M,N", SHAPES + [(2600, 4100)])
@pytest.mark.parametrize("af,bf,br", [("e4m3", "e4m3", 128), ("e5m2", "e4m3", 1)])
def test_block128(af, bf, br, M, N):
    for K in DEPTHS:
        say(f"ones: block128 {af} {bf} {M} x {N} x {K}")
        a, b = ones((M, K), ONE[af]), ones((N, K), ONE[bf])
        sa, sb = ones(bs.block128_scale_shape(M, K, 1), 127), ones(bs.block128_scale_shape(N, K, br), 127)
        check(lambda out, alpha, c, beta: bs.scaled_gemm_block128(a, sa, b, sb, af, bf, 1, br, out=out, alpha=alpha, c=c, beta=beta),
              M, N, K, f"block128 {af} {bf} {M} x {N} x {K}")


#: groups' sizes (with walks of several 16-row tiles on the form for few rows) and columns
GROUPED = [([0] * 30 + [203, 17] + [1] * 22, 16), ([3, 0, 20, 1], 1000), ([700, 0, 1, 300], 520), ([2000, 1, 1500], 1001),
           ([3001, 0, 2999], 4096)]


@pytest.mark.parametrize("sizes,N", GROUPED)
@pytest.mark.parametrize("af,bf", [("e4m3", "e4m3"), ("e5m2", "e4m3")])
def test_grouped(af, bf, sizes, N):
    import torch
    M, E = sum(sizes), len(sizes)
    o = torch.tensor([sum(sizes[:i]) for i in range(E + 1)], dtype=torch.int32, device="cuda")
    for K in DEPTHS:
        say(f"ones: grouped {af} {bf} {E} groups {M} x {N} x {K}")
        a, b = ones((M, K), ONE[af]), ones((E, N, K), ONE[bf])
        sa, sb = ones(bs.block128_scale_shape(M, K, 1), 127), ones((E, *bs.block128_scale_shape(N, K, 128)), 127)
        check(lambda out, alpha, c, beta: bs.scaled_gemm_grouped_block128(a, sa, b, sb, o, af, bf, 128, out, alpha, c, beta),
              M, N, K, f"grouped {af} {bf} {E} groups {M} x {N} x {K}")


@pytest.mark.parametrize("rows,E,M,N", [(32, 4, 96, 130), (160, 3, 700, 1001), (512, 5, 300, 64), (2048, 3, 2000, 2050)])
@pytest.mark.parametrize("af,bf", [("e4m3", "e4m3"), ("e5m2", "e4m3")])
def test_weight_gradient(af, bf, rows, E, M, N):
    """Groups of the same size, so that every element of every group is that size; a group without rows among them."""
    import torch
    sizes = [rows] * E
    sizes[1] = 0
    n = sum(sizes)
    o = torch.tensor([sum(sizes[:i]) for i in range(E + 1)], dtype=torch.int32, device="cuda")
    say(f"ones: weight gradient {af} {bf} {sizes} {M} x {N}")
    parts = [bs.fp8_quantize_grouped_block128(torch.ones((n, w), device="cuda"), o, f, rows=False, transposed=True)
             for w, f in ((M, af), (N, bf))]
    (a, sa), (b, sb) = parts
    for out, dt in (("f32", torch.float32), ("bf16", torch.bfloat16), ("f16", torch.float16)):
        for alpha, beta in EPILOGUES:
            c = None if beta == 0.0 else torch.full((E, M, N), -16.0, dtype=dt, device="cuda")
            d = bs.scaled_gemm_grouped_wgrad_block128(a, sa, b, sb, o, af, bf, out, alpha, c, beta)
            for e in range(E):
                want = alpha * sizes[e] + (0.0 if c is None else beta * -16.0)
                wrong = int((d[e].double() != want).sum())
                assert wrong == 0, f"{out} alpha {alpha} beta {beta} group {e}: {wrong} elements are not {want}"
