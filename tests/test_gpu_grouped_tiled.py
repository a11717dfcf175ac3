"""What the grouped products promise beside their values, on the tiled forms (MI355X): nothing written outside D's
elements, C and D the same array, alpha with beta, offsets that break the rules, captured calls that follow
new offsets, and outputs past 2^32 bytes.  The form is asked of the library.  Tolerances as in test_gpu_grouped.py.
"""
import numpy as np
import pytest

import block_scaled_precision_fp8_amd as bs
from gpu_common import guarded, say, untouched
from test_gpu_grouped import dtype, offs
from test_gpu_grouped_forms import _check, _random, _values
from test_gpu_grouped_narrow import columns_form, rows_form

pytestmark = pytest.mark.gpu

BITS = {4: "int32", 2: "int16"}


def bits(t):
    import torch
    return t.contiguous().view(getattr(torch, BITS[t.element_size()]))


def row_operands(sizes, N, K, i, first=2, after=3):
    """Codes and scales of a product by rows, its offsets, formats and block rows."""
    import torch
    o, od = offs(sizes, first=first)
    M = int(o[-1]) + after
    af, bf, br = ("e4m3", "e5m2")[i % 2], ("e4m3", "e5m2")[i // 2 % 2], (128, 1)[i % 2]
    a, sa = bs.fp8_quantize_block128(_random((M, K), i), af)
    b = torch.empty((len(sizes), N, K), dtype=torch.uint8, device="cuda")
    sb = torch.empty((len(sizes), *bs.block128_scale_shape(N, K, br)), dtype=torch.uint8, device="cuda")
    for e in range(len(sizes)):
        bs.fp8_quantize_block128(_random((N, K), 50 + e), bf, br, codes=b[e], scales=sb[e])
    return M, o, od, (a, sa, b, sb), (af, bf, br)


def column_operands(sizes, M, N, i):
    o, od = offs(sizes)
    af, bf = ("e5m2", "e4m3")[i % 2], ("e4m3", "e5m2")[i // 2 % 2]
    a, sa = bs.fp8_quantize_grouped_block128(_random((int(o[-1]), M), i), od, af, rows=False, transposed=True)
    b, sb = bs.fp8_quantize_grouped_block128(_random((int(o[-1]), N), 20 + i), od, bf, rows=False, transposed=True)
    return o, od, (a, sa, b, sb), (af, bf)


#: form, output, sizes, N, K, alpha, beta
ROWS = [
    ("T64x128", "bf16", [40, 0, 64, 65, 1, 30, 128, 17, 20, 25, 40, 60, 31, 33, 20, 26], 1001, 1056, -2.0, 0.5),
    ("T64x128", "f16", [40, 0, 64, 65, 1, 30, 128, 17, 20, 25, 40, 60, 31, 33, 20, 26], 1003, 544, 0.5, 0.0),
    ("T64x128", "f32", [100, 20, 0, 180, 64, 36], 2050, 992, -2.0, 0.5),
    ("T128", "bf16", [2000, 1, 0, 1500, 2499], 1003, 1056, -2.0, 0.5),
    ("T128", "f16", [2000, 1, 0, 1500, 2499], 1001, 1024, 0.5, 0.0),
    ("T128", "f32", [1999, 129, 0, 2500, 1372], 1001, 1056, -2.0, 0.5),
    ("T256", "bf16", [3001, 0, 257, 2742], 4093, 4064, -2.0, 0.0),
    ("T256", "f16", [2999, 1, 3000], 4099, 4096, 0.5, 0.0),
]
#: form, output, sizes, M, N, alpha, beta
COLUMNS = [
    ("T128", "bf16", [100, 0, 300, 17, 1000, 130], 700, 1001, -2.0, 0.5),
    ("T128", "f16", [100, 0, 300, 17, 1000, 130], 701, 1003, 0.5, 0.0),
    ("T128", "f32", [900, 0, 300, 17, 1000, 130], 641, 901, -2.0, 0.5),
    ("T256", "bf16", [2600, 0, 3401], 2001, 2049, -2.0, 0.0),
    ("T256", "f16", [129, 3000, 0, 2500], 3901, 4093, 0.5, 0.0),
    ("T256", "f32", [3300, 0, 129, 2571], 4096, 4096, 1.0, 1.0),
    ("T256", "f32", [3300, 0, 129, 2571], 4095, 4091, -2.0, 0.5),
]


@pytest.mark.parametrize("extra", [0, 3, 8])
@pytest.mark.parametrize("case", ROWS, ids=lambda c: f"{c[0]}-{c[1]}-{c[3]}")
def test_rows(case, extra):
    import torch
    form, out, sizes, N, K, alpha, beta = case
    label = f"grouped {form} {out} {sizes[:6]} N {N} K {K} alpha {alpha} beta {beta} extra {extra}"
    say(label)
    M, o, od, ops, fmts = row_operands(sizes, N, K, ROWS.index(case))
    assert rows_form(M, N, K, len(sizes), out, N + extra, N if beta else 0, beta) == form
    c = _random((M, N), 99).to(dtype(out)) if beta else None
    buf, d = guarded((M, N), dtype(out), extra_cols=extra, extra_rows=1, tail=64)
    before = d.clone()
    bs.scaled_gemm_grouped_block128(*ops, od, *fmts, out=out, alpha=alpha, c=c, beta=beta, d=d)
    assert untouched(buf, (M, N), extra, 1, 64)
    for part in (slice(0, 2), slice(M - 3, M)):
        assert bits(d[part]).equal(bits(before[part]))
    for e in np.flatnonzero(sizes):
        p, q = int(o[e]), int(o[e + 1])
        x, y = _values(ops[0][p:q], ops[1][:, p:q], fmts[0]), _values(ops[2][e], ops[3][e], fmts[1], fmts[2])
        _check(d[p:q], x @ y.t().contiguous(), x.abs() @ y.abs().t().contiguous(), out, K, alpha,
               None if c is None else beta * c[p:q].double(), f"{label} group {e}")
    if beta:
        same, d2 = guarded((M, N), dtype(out), extra_cols=extra, extra_rows=1, tail=64)
        d2.copy_(c)
        assert rows_form(M, N, K, len(sizes), out, N + extra, N + extra, beta) == form
        bs.scaled_gemm_grouped_block128(*ops, od, *fmts, out=out, alpha=alpha, c=d2, beta=beta, d=d2)
        assert bits(d2[2:M - 3]).equal(bits(d[2:M - 3])) and untouched(same, (M, N), extra, 1, 64)
        assert d2[:2].equal(c[:2]) and d2[M - 3:].equal(c[M - 3:])


@pytest.mark.parametrize("extra", [0, 3, 8])
@pytest.mark.parametrize("case", COLUMNS, ids=lambda c: f"{c[0]}-{c[1]}-{c[4]}")
def test_columns(case, extra):
    """Matrices one row apart in a buffer of canaries, rows `extra` elements apart."""
    import torch
    form, out, sizes, M, N, alpha, beta = case
    label = f"wgrad {form} {out} {sizes[:6]} M {M} N {N} alpha {alpha} beta {beta} extra {extra}"
    say(label)
    E = len(sizes)
    o, od, ops, fmts = column_operands(sizes, M, N, COLUMNS.index(case))
    columns = ops[0].shape[1]
    assert columns_form(M, N, columns, E, out, N + extra, N if beta else 0, beta) == form

    def room():
        buf, flat = guarded((E * (M + 1), N), dtype(out), extra_cols=extra, extra_rows=1, tail=64)
        return buf, flat.unflatten(0, (E, M + 1))

    def whole(buf, v, edge):
        return untouched(buf, (E * (M + 1), N), extra, 1, 64) and bits(v[:, M]).equal(edge)

    c = _random((E * M, N), 99).view(E, M, N).to(dtype(out)) if beta else None
    buf, v = room()
    d, edge = v[:, :M], bits(v[:, M])
    bs.scaled_gemm_grouped_wgrad_block128(*ops, od, *fmts, out=out, alpha=alpha, c=c, beta=beta, d=d)
    assert whole(buf, v, edge)
    col = word = 0
    for e, n in enumerate(sizes):
        end, last = col + (n + 127) // 128 * 128, word + (n + 511) // 512
        if n:
            x, y = _values(ops[0][:, col:end], ops[1][word:last], fmts[0]), _values(ops[2][:, col:end], ops[3][word:last], fmts[1])
            want, s = x @ y.t().contiguous(), x.abs() @ y.abs().t().contiguous()
        else:
            want = s = torch.zeros((M, N), dtype=torch.float64, device="cuda")
        _check(d[e], want, s, out, n + 128, alpha, None if c is None else beta * c[e].double(), f"{label} group {e}")
        col, word = end, last
    if beta:
        same, w = room()
        w[:, :M] = c
        assert columns_form(M, N, columns, E, out, N + extra, N + extra, beta) == form
        bs.scaled_gemm_grouped_wgrad_block128(*ops, od, *fmts, out=out, alpha=alpha, c=w[:, :M], beta=beta, d=w[:, :M])
        assert bits(w[:, :M]).equal(bits(d)) and whole(same, w, edge)


#: of 6000 rows and four groups
BROKEN = [[0, 4000, 100, 5000, 6000], [-7, 30, 60, 90, 6000], [0, 20000, 30000, 40000, 50000], [6000, 4000, 3000, 2000, 0],
          [5, 5, 5, 5, 5], [0, 2 ** 31 - 1, -(2 ** 31), 6000, 90], [-5, -4, -3, -2, -1], [5990, 6050, 6100, 7000, 7001],
          [0, 6000, 12000, 18000, 24000]]


@pytest.mark.parametrize("form,out,N,K", [("T64x128", "bf16", 70, 1056), ("T64x128", "f32", 130, 544), ("T128", "bf16", 1003, 1024),
                                          ("T128", "f32", 1001, 1024), ("T256", "bf16", 4093, 4064), ("T256", "f16", 4096, 4096)])
def test_rows_by_offsets_that_break_the_rules(form, out, N, K):
    """Nothing outside D's elements is written (what is inside is undefined), and a call with proper offsets
    afterwards gives what it gave before."""
    import torch
    sizes = [2500, 0, 1700, 1800]
    M, o, od, ops, fmts = row_operands(sizes, N, K, 1, first=0, after=0)
    assert M == 6000 and rows_form(M, N, K, 4, out, N + 3) == form
    proper = bs.scaled_gemm_grouped_block128(*ops, od, *fmts, out=out)
    buf, d = guarded((M, N), dtype(out), extra_cols=3, extra_rows=300, tail=4096)
    for bad in BROKEN:
        say(f"grouped {form} {out} offsets {bad}")
        t = torch.tensor(bad, dtype=torch.int32, device="cuda")
        bs.scaled_gemm_grouped_block128(*ops, t, *fmts, out=out, d=d)
        assert untouched(buf, (M, N), 3, 300, 4096)
    bs.scaled_gemm_grouped_block128(*ops, od, *fmts, out=out, d=d)
    assert d.equal(proper)


@pytest.mark.parametrize("form,out,M,N", [("T128", "bf16", 700, 1001), ("T128", "f32", 641, 901), ("T256", "bf16", 4001, 4093),
                                          ("T256", "f32", 4095, 4091)])
def test_columns_by_offsets_that_break_the_rules(form, out, M, N):
    import torch
    o, od, ops, fmts = column_operands([2500, 0, 1700, 1800], M, N, 1)
    assert int(o[-1]) == 6000 and columns_form(M, N, ops[0].shape[1], 4, out, N + 3) == form
    proper = bs.scaled_gemm_grouped_wgrad_block128(*ops, od, *fmts, out=out)
    buf, flat = guarded((4 * M, N), dtype(out), extra_cols=3, extra_rows=300, tail=4096)
    d = flat.unflatten(0, (4, M))
    for bad in BROKEN:
        say(f"wgrad {form} {out} offsets {bad}")
        t = torch.tensor(bad, dtype=torch.int32, device="cuda")
        bs.scaled_gemm_grouped_wgrad_block128(*ops, t, *fmts, out=out, d=d)
        assert untouched(buf, (4 * M, N), 3, 300, 4096)
    bs.scaled_gemm_grouped_wgrad_block128(*ops, od, *fmts, out=out, d=d)
    assert d.equal(proper)


@pytest.mark.parametrize("form,out,N,K", [("T64x128", "bf16", 70, 1056), ("T128", "f32", 1001, 1024), ("T256", "bf16", 4093, 4064)])
def test_captured_rows_follow_new_offsets(form, out, N, K):
    import torch
    say(f"a captured {form} product by rows")
    M, o, od, ops, fmts = row_operands([2500, 0, 1700, 1800], N, K, 0, first=0, after=0)
    assert rows_form(M, N, K, 4, out) == form
    # (rows of no group are left as they were: D starts as it does for the eager call)
    d = torch.zeros((M, N), dtype=dtype(out), device="cuda")
    run = lambda to: bs.scaled_gemm_grouped_block128(*ops, od, *fmts, out=out, d=to)       # noqa: E731
    graph = capture(lambda: run(d))
    for new in ([0, 2500, 2500, 4200, 6000], [0, 0, 0, 0, 6000], [0, 1, 129, 130, 5000], [1000, 3000, 3001, 3001, 5999]):
        od.copy_(torch.tensor(new, dtype=torch.int32))
        d.zero_()
        graph.replay()
        want = torch.zeros_like(d)
        run(want)
        assert d.equal(want), new


@pytest.mark.parametrize("form,out,M,N", [("T128", "bf16", 700, 1001), ("T256", "f32", 4095, 4091)])
def test_captured_columns_follow_new_offsets(form, out, M, N):
    """With the quantisers that lay the operands out, and added to what is there."""
    import torch
    say(f"a captured {form} weight gradient")
    o, od = offs([2500, 0, 1700, 1800])
    x, y = _random((6000, M), 1), _random((6000, N), 2)
    beta = 1.0 if out == "f32" else 0.0
    start = _random((4 * M, N), 3).view(4, M, N).to(dtype(out))

    def run(to):
        a, sa = bs.fp8_quantize_grouped_block128(x, od, "e5m2", rows=False, transposed=True)
        b, sb = bs.fp8_quantize_grouped_block128(y, od, "e4m3", rows=False, transposed=True)
        assert columns_form(M, N, a.shape[1], 4, out, N, N if beta else 0, beta) == form
        return bs.scaled_gemm_grouped_wgrad_block128(a, sa, b, sb, od, "e5m2", "e4m3", out=out, c=to if beta else None,
                                                     beta=beta, d=to)

    d = start.clone()
    graph = capture(lambda: run(d))
    for new in ([0, 2500, 2500, 4200, 6000], [0, 0, 0, 0, 6000], [0, 1, 129, 130, 6000], [0, 3000, 3001, 3001, 5999]):
        od.copy_(torch.tensor(new, dtype=torch.int32))
        d.copy_(start)
        graph.replay()
        assert d.equal(run(start.clone())), new


def capture(run):
    import torch
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    return graph


# ------------------------------------------------------------------ past 2^32 bytes
def test_transposed_codes_past_32_bits():
    """A transpose of more than 2^32 bytes of codes: its last rows and columns against their own small call."""
    say("quantize_grouped: codes of the transpose past 2^32 bytes")
    k, sizes = 40000, [60000, 0, 51000, 300]
    o, od = offs(sizes)
    x = _random((int(o[-1]), k), 1).bfloat16()
    q, s = bs.fp8_quantize_grouped_block128(x, od, "e4m3", rows=False, transposed=True)
    assert q.numel() > 1 << 32
    col, word = sum((n + 127) // 128 * 128 for n in sizes[:3]), sum((n + 511) // 512 for n in sizes[:3])
    part = x[-300:, k - 260:].contiguous()
    want, ws = bs.fp8_quantize_grouped_block128(part, offs([300])[1], "e4m3", rows=False, transposed=True)
    assert q[k - 260:, col:col + 384].equal(want[:, :384]) and s[word:word + 1, k - 260:].equal(ws[:1])


@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_weight_gradients_past_32_bits(out):
    """D of more than 2^32 bytes, in place for FP32: the last group against float64."""
    import torch
    E, M, N = 36, 8192, 8200
    say(f"weight gradients past 2^32 bytes, {out}")
    sizes = [40] * E
    sizes[3], sizes[-1] = 0, 300
    o, od, ops, fmts = column_operands(sizes, M, N, 1)
    beta = 1.0 if out == "f32" else 0.0
    d = torch.full((E, M, N), 5.0, dtype=dtype(out), device="cuda")
    assert d.numel() * d.element_size() > 1 << 32
    assert columns_form(M, N, ops[0].shape[1], E, out, N, N if beta else 0, beta) == "T256"
    bs.scaled_gemm_grouped_wgrad_block128(*ops, od, *fmts, out=out, c=d if beta else None, beta=beta, d=d)
    col, word = sum((n + 127) // 128 * 128 for n in sizes[:-1]), sum((n + 511) // 512 for n in sizes[:-1])
    x = _values(ops[0][-600:, col:col + 384], ops[1][word:word + 1, -600:], fmts[0])
    y = _values(ops[2][-600:, col:col + 384], ops[3][word:word + 1, -600:], fmts[1])
    _check(d[-1, -600:, -600:], x @ y.t().contiguous(), x.abs() @ y.abs().t().contiguous(), out, 428, 1.0,
           torch.full((600, 600), 5.0, device="cuda") if beta else None, "last group")
    assert bool((d[3] == (5.0 if beta else 0.0)).all())
