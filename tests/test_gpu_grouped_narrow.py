"""Products by expert with few columns: which kernel form they run on, asked of the library itself (CPU), and their
results against float64 (MI355X).

The form for few rows has one workgroup per 16 columns and group, which walks its group's rows 16 at a time.  With many
rows to a group and few columns to share them, that walk is the whole time: 16384 rows of 8 groups, N = 16,
K = 4096 took 557 us there and 19 on tiles of 64 x 128.
"""
import ctypes

import numpy as np
import pytest

import block_scaled_precision_fp8_amd as bs
from gpu_common import say, untouched, guarded
from test_gpu_grouped import dtype, offs
from test_gpu_grouped_forms import COLUMNS, ROWS, _check, _random, _values, fast

NAMES = ("FEW", "T64x128", "T128", "T256")
OUTS = ("f32", "bf16", "f16")
i64, c_int = ctypes.c_int64, ctypes.c_int


def rows_form(M, N, K, groups, out="bf16", ldd=None, ldc=0, beta=0.0):
    f = bs.lib()._ZN5bsfp817gemm_grouped_formEllliillf
    f.argtypes, f.restype = [i64, i64, i64, c_int, c_int, i64, i64, ctypes.c_float], c_int
    return NAMES[f(M, N, K, groups, OUTS.index(out), N if ldd is None else ldd, ldc, beta)]


def columns_form(M, N, columns, groups, out="bf16", ldd=None, ldc=0, beta=0.0):
    f = bs.lib()._ZN5bsfp815gemm_wgrad_formEllliillf
    f.argtypes, f.restype = [i64, i64, i64, c_int, c_int, i64, i64, ctypes.c_float], c_int
    return NAMES[f(M, N, columns, groups, OUTS.index(out), N if ldd is None else ldd, ldc, beta)]


def c_of(epilogue, N):
    return dict(beta=1.0, ldc=N) if epilogue == "c" else {}


@pytest.mark.parametrize("form,out,sizes,N,K,epilogue", ROWS)
def test_rows_cases_run_on_their_form(form, out, sizes, N, K, epilogue):
    """The library's own choice, with the rows that belong to no group (5 of them) counted."""
    assert rows_form(sum(sizes) + 5, N, K, len(sizes), out, **c_of(epilogue, N)) == form


@pytest.mark.parametrize("form,out,sizes,M,N,epilogue", COLUMNS)
def test_columns_cases_run_on_their_form(form, out, sizes, M, N, epilogue):
    columns = bs.lib().block128_grouped_columns(sum(sizes), len(sizes))
    assert columns_form(M, N, columns, len(sizes), out, **c_of(epilogue, N)) == form


def test_strides_and_c_keep_calls_off_the_largest_tile():
    assert rows_form(16384, 14336, 4096, 8) == "T256"
    for kw in (dict(ldd=1 << 21), dict(beta=1.0, ldc=14336), dict(out="f32")):
        assert rows_form(16384, 14336, 4096, 8, **kw) != "T256"
    columns = bs.lib().block128_grouped_columns(16384, 8)
    assert columns_form(4096, 4096, columns, 8) == columns_form(4096, 4096, columns, 8, "f32", beta=1.0, ldc=4096) == "T256"
    for kw in (dict(ldd=1 << 21), dict(beta=1.0, ldc=4096), dict(out="f32", beta=1.0, ldc=1 << 21)):
        assert columns_form(4096, 4096, columns, 8, **kw) != "T256"


#: rows, groups, N, K, output and the measured microseconds (few rows, 64 x 128), groups of equal shares
MEASURED = [(16384, 8, 16, 4096, "bf16", 557, 19.3), (16384, 8, 3, 4096, "bf16", 422, 19.6),
            (16384, 2, 3, 512, "bf16", 427, 6.1), (11780, 2, 3, 4096, "bf16", None, None),
            (2048, 2, 48, 4096, "bf16", 281, 14.7), (2048, 8, 16, 512, "bf16", 14.7, 4.6),
            (512, 2, 128, 4096, "bf16", 73, 12.4), (128, 2, 16, 4096, "bf16", 21, 12.2),
            (16384, 64, 3, 4096, "bf16", 61.5, 19.7), (16384, 2, 8, 4096, "f32", 1950, 28.5)]
SHORT = [(128, 8, 16, 4096, "bf16", 8.9, 12.3), (128, 8, 16, 512, "bf16", 2.9, 4.4), (128, 64, 128, 4096, "bf16", 9.3, 15.6),
         (512, 64, 16, 4096, "bf16", 5.8, 12.3), (512, 64, 48, 512, "bf16", 2.4, 4.5), (8, 16, 1024, 4096, "bf16", 8.6, 15.9)]


@pytest.mark.parametrize("M,groups,N,K,out,few,tiled", MEASURED)
def test_long_walks_run_on_tiles(M, groups, N, K, out, few, tiled):
    assert few is None or few > 1.5 * tiled
    assert rows_form(M, N, K, groups, out) in ("T64x128", "T128")


@pytest.mark.parametrize("M,groups,N,K,out,few,tiled", SHORT)
def test_short_walks_stay(M, groups, N, K, out, few, tiled):
    assert few < tiled and rows_form(M, N, K, groups, out) == "FEW"


#: equal shares, all rows in one group, and walks of several tiles on the form for few rows
SIZES = [([300] * 7 + [301], 3, 1056, "bf16", "plain"), ([0, 2400, 1], 8, 544, "f16", "alpha"), ([700, 900], 16, 512, "f32", "c"),
         ([1500, 0], 1, 512, "bf16", "c"), ([0] * 40 + [203, 17] + [1] * 22, 16, 1056, "bf16", "plain"),
         ([0] * 40 + [130, 49] + [0] * 22, 33, 544, "f32", "c")]


@pytest.mark.gpu
@pytest.mark.parametrize("sizes,N,K,out,epilogue", SIZES)
def test_few_columns(sizes, N, K, out, epilogue):
    import torch
    label = f"grouped {len(sizes)} groups up to {max(sizes)} rows N {N} K {K} {out} {epilogue}"
    say(label)
    o, od = offs(sizes, first=2)
    M, E, i = int(o[-1]) + 3, len(sizes), SIZES.index((sizes, N, K, out, epilogue))
    assert (rows_form(M, N, K, E, out, **c_of(epilogue, N)) == "FEW") == (E > 50)
    af, bf, br = ("e4m3", "e5m2")[i % 2], ("e4m3", "e5m2")[i // 2 % 2], (128, 1)[i % 2]
    a, sa = bs.fp8_quantize_block128(_random((M, K), i), af)
    w = [bs.fp8_quantize_block128(_random((N, K), 50 + e), bf, br) for e in range(E)]
    b, sb = (torch.stack(t) for t in zip(*w))
    alpha = -0.75 if epilogue == "alpha" else 1.0
    c = _random((M, N), 99).to(dtype(out)) if epilogue == "c" else None
    buf, d = guarded((M, N), dtype(out), extra_cols=3, extra_rows=1, tail=16)
    before = d.clone()
    bs.scaled_gemm_grouped_block128(a, sa, b, sb, od, af, bf, br, out=out, alpha=alpha, c=c, beta=0.0 if c is None else 1.0, d=d)
    bits = {4: torch.int32, 2: torch.int16}[d.element_size()]
    for part in (slice(0, 2), slice(M - 3, M)):
        assert d[part].contiguous().view(bits).equal(before[part].contiguous().view(bits))
    assert untouched(buf, (M, N), 3, 1, 16)
    for e in np.flatnonzero(sizes):
        p, q = int(o[e]), int(o[e + 1])
        x, y = _values(a[p:q], sa[:, p:q], af), _values(b[e], sb[e], bf, br)
        _check(d[p:q], x @ y.t().contiguous(), x.abs() @ y.abs().t().contiguous(), out, K, alpha,
               None if c is None else c[p:q], f"{label} group {e}")
