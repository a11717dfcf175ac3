"""Every form of the grouped products, with one and with several tiles per workgroup, ragged and empty
groups and partial tiles, against float64 products of the dequantised operands (MI355X).  Tolerances as
in test_gpu_grouped.py.  The first tests (CPU) check that the cases reach the forms they are for."""
import numpy as np
import pytest

import block_scaled_precision_fp8_amd as bs
from gpu_common import say
from grouped_forms import columns_form, costs, rows_form
from test_gpu_grouped import TINY, dtype, offs, tol

# form, output, sizes of groups, N, K, epilogue
ROWS = [
    ("FEW", "bf16", [1, 0, 3, 20, 1, 2, 0, 5], 1000, 1056, "plain"),
    ("FEW", "f32", [2, 1, 4, 1], 520, 2080, "c"),
    ("T64x128", "bf16", [40, 0, 64, 65, 1, 30, 128, 17, 20, 25, 40, 60, 31, 33, 20, 26], 1024, 1024, "plain"),
    ("T64x128", "f16", [40, 0, 64, 65, 1, 30, 128, 17, 20, 25, 40, 60, 31, 33, 20, 26], 1001, 1056, "c"),
    ("T64x128", "f32", [100, 20, 0, 180, 64, 36], 2052, 992, "alpha"),
    ("T128", "bf16", [2000, 1, 0, 1500, 2499], 1000, 1024, "alpha"),
    ("T128", "bf16", [2000, 1, 0, 1500, 2499], 999, 1088, "c"),
    ("T128", "f32", [1999, 129, 0, 2500, 1372], 1004, 1024, "c"),
    ("T256", "bf16", [3001, 0, 257, 2742], 4096, 4096, "plain"),
    ("T256", "f16", [2999, 1, 3000], 4088, 4064, "alpha"),
    ("T256", "bf16", [2999, 1, 3000], 4093, 4096, "plain"),
]
# form, output, sizes, M, N, epilogue
COLUMNS = [
    ("FEW", "bf16", [500, 0, 3, 1200], 96, 130, "plain"),
    ("FEW", "f32", [129, 127, 0, 1], 100, 70, "c"),
    ("T128", "bf16", [100, 0, 300, 17, 1000, 130], 700, 1001, "c"),
    ("T128", "f16", [100, 0, 300, 17, 1000, 130], 700, 1000, "plain"),
    ("T128", "f32", [900, 0, 300, 17, 1000, 130], 640, 900, "c"),
    ("T128", "f32", [900, 0, 300, 17, 1000, 130], 640, 901, "alpha"),
    ("T256", "bf16", [2600, 0, 3401], 2000, 2048, "plain"),
    ("T256", "f16", [129, 3000, 0, 2500], 3900, 4096, "alpha"),
    ("T256", "f32", [3300, 0, 129, 2571], 4096, 4092, "c"),
    ("T256", "f32", [3300, 0, 129, 2571], 4096, 4091, "c"),
    ("T256", "bf16", [69] * 20, 1000, 2001, "plain"),
]


def fast(out, N, epilogue):
    return out == "f32" or epilogue != "c"


@pytest.mark.parametrize("form,out,sizes,N,K,epilogue", ROWS)
def test_rows_cases_reach_their_form(form, out, sizes, N, K, epilogue):
    assert rows_form(sum(sizes), N, K, len(sizes), out == "f32", fast(out, N, epilogue)) == form


@pytest.mark.parametrize("form,out,sizes,M,N,epilogue", COLUMNS)
def test_columns_cases_reach_their_form(form, out, sizes, M, N, epilogue):
    columns = bs.lib().block128_grouped_columns(sum(sizes), len(sizes))
    assert columns_form(M, N, columns, len(sizes), out == "f32", fast(out, N, epilogue)) == form


def test_every_form_has_cases():
    names = {n for n, *_ in costs()} | {"FEW"}
    assert {c[0] for c in ROWS} == names and {c[0] for c in COLUMNS} == names - {"T64x128"}


def _values(codes, scales, fmt, rows=1):
    """float64 values of codes and scale words, on the device."""
    import torch
    f8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}[fmt]
    s = scales.transpose(0, 1).reshape(scales.shape[1], -1).double()
    s = torch.exp2(s - 127).repeat_interleave(rows, 0)[:codes.shape[0]].repeat_interleave(128, 1)[:, :codes.shape[1]]
    return codes.view(f8).double() * s


def _random(shape, seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rows = torch.exp2(torch.randint(-4, 5, (shape[0], 1), generator=g, device="cuda").float())
    return torch.randn(shape, generator=g, device="cuda") * rows


def _check(d, want, s, out, K, alpha, c, label):
    r, m = alpha * want, abs(alpha) * s
    if c is not None:
        r, m = r + c.double(), m + c.double().abs()
    lim = tol(out, K) * m + TINY[out]
    err = (d.double() - r).abs()
    if out == "f16":
        over = d.isinf() & (r.abs() + lim >= 65520) & (d.sign() == r.sign())
        err = err.masked_fill(over, 0.0)
    worst = float((err / lim.clamp(min=1e-300)).max())
    say(f"{label}: {worst:.3f} of the bound")
    assert bool((err <= lim).all()), f"{label}: {worst:.3f} of the bound"


@pytest.mark.gpu
@pytest.mark.parametrize("form,out,sizes,N,K,epilogue", ROWS)
def test_rows(form, out, sizes, N, K, epilogue):
    import torch
    label = f"grouped {form} {out} {sizes[:6]} N {N} K {K} {epilogue}"
    say(label)
    E, (o, od) = len(sizes), offs(sizes, first=2)
    M = int(o[-1]) + 3
    i = ROWS.index((form, out, sizes, N, K, epilogue))
    af, bf, br = ("e4m3", "e5m2")[i % 2], ("e4m3", "e5m2")[i // 2 % 2], (128, 1)[i // 3 % 2]
    a, sa = bs.fp8_quantize_block128(_random((M, K), i), af)
    b = torch.empty((E, N, K), dtype=torch.uint8, device="cuda")
    sb = torch.empty((E, *bs.block128_scale_shape(N, K, br)), dtype=torch.uint8, device="cuda")
    for e in range(E):
        bs.fp8_quantize_block128(_random((N, K), 50 + e), bf, br, codes=b[e], scales=sb[e])
    alpha = -0.75 if epilogue == "alpha" else 1.0
    c = _random((M, N), 99).to(dtype(out)) if epilogue == "c" else None
    d = torch.full((M, N), 7.0, dtype=dtype(out), device="cuda")
    bs.scaled_gemm_grouped_block128(a, sa, b, sb, od, af, bf, br, out=out, alpha=alpha, c=c, beta=0.0 if c is None else 1.0, d=d)
    assert bool((d[:2] == 7.0).all()) and bool((d[-3:] == 7.0).all())
    for e in range(E):
        p, q = int(o[e]), int(o[e + 1])
        if p < q:
            x, y = _values(a[p:q], sa[:, p:q], af), _values(b[e], sb[e], bf, br)
            _check(d[p:q], x @ y.t().contiguous(), x.abs() @ y.abs().t().contiguous(), out, K, alpha,
                   None if c is None else c[p:q], f"{label} group {e}")


@pytest.mark.gpu
@pytest.mark.parametrize("form,out,sizes,M,N,epilogue", COLUMNS)
def test_columns(form, out, sizes, M, N, epilogue):
    import torch
    label = f"wgrad {form} {out} {sizes[:6]} M {M} N {N} {epilogue}"
    say(label)
    E, (o, od) = len(sizes), offs(sizes)
    i = COLUMNS.index((form, out, sizes, M, N, epilogue))
    af, bf = ("e5m2", "e4m3")[i % 2], ("e4m3", "e5m2")[i // 2 % 2]
    a, sa = bs.fp8_quantize_grouped_block128(_random((int(o[-1]), M), i), od, af, rows=False, transposed=True)
    b, sb = bs.fp8_quantize_grouped_block128(_random((int(o[-1]), N), 20 + i), od, bf, rows=False, transposed=True)
    alpha = -0.75 if epilogue == "alpha" else 1.0
    c = _random((E * M, N), 99).view(E, M, N).to(dtype(out)) if epilogue == "c" else None
    d = bs.scaled_gemm_grouped_wgrad_block128(a, sa, b, sb, od, af, bf, out=out, alpha=alpha, c=c,
                                              beta=0.0 if c is None else 1.0)
    col = word = 0
    for e, n in enumerate(sizes):
        end, last = col + (n + 127) // 128 * 128, word + (n + 511) // 512
        if n:
            x, y = _values(a[:, col:end], sa[word:last], af), _values(b[:, col:end], sb[word:last], bf)
            want, s = x @ y.t().contiguous(), x.abs() @ y.abs().t().contiguous()
        else:
            want = s = torch.zeros((M, N), dtype=torch.float64, device="cuda")
        _check(d[e], want, s, out, n + 128, alpha, None if c is None else c[e], f"{label} group {e}")
        col, word = end, last


@pytest.mark.gpu
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_rows_of_outputs_further_apart_than_32_bit_offsets_reach(out):
    """Row strides of 2^21 elements and more take the epilogue with 64-bit addresses."""
    import torch
    ld, sizes, N, K = (1 << 21) + 8, [100, 20, 0, 180, 64, 36], 2052, 992
    say(f"outputs with a row stride of {ld} elements, {out}")
    o, od = offs(sizes)
    M = int(o[-1])
    assert rows_form(M, N, K, len(sizes), out == "f32", False) == "T64x128"
    a, sa = bs.fp8_quantize_block128(_random((M, K), 1))
    w = [bs.fp8_quantize_block128(_random((N, K), 2 + e), "e4m3", 128) for e in range(len(sizes))]
    b, sb = (torch.stack(t) for t in zip(*w))
    d = torch.empty((M, ld), dtype=dtype(out), device="cuda")[:, :N]
    bs.scaled_gemm_grouped_block128(a, sa, b, sb, od, out=out, d=d)
    assert d.equal(bs.scaled_gemm_grouped_block128(a, sa, b, sb, od, out=out))
    sizes, M, N = [500, 800], 1300, 900
    o, od = offs(sizes)
    columns = bs.lib().block128_grouped_columns(int(o[-1]), 2)
    assert columns_form(M, N, columns, 2, out == "f32", False) == "T128"
    x, sx = bs.fp8_quantize_grouped_block128(_random((1300, M), 3), od, rows=False, transposed=True)
    y, sy = bs.fp8_quantize_grouped_block128(_random((1300, N), 4), od, rows=False, transposed=True)
    g = torch.empty((2, M, ld), dtype=dtype(out), device="cuda")[:, :, :N]
    bs.scaled_gemm_grouped_wgrad_block128(x, sx, y, sy, od, out=out, d=g)
    assert g.equal(bs.scaled_gemm_grouped_wgrad_block128(x, sx, y, sy, od, out=out))
