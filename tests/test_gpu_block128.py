"""Parity of the block-of-128 FP8 quantiser and GEMM with their float64 references (MI355X).

Quantiser: byte-equal.  GEMM: |D - D_ref| <= tol(K) (|alpha| S + |beta C|), S = sum |a b|, where
tol follows from the matrix instructions' arithmetic and counts worst cases:
  16-bit outputs: the FP8 instruction cuts each group of 8 products to 13 fraction bits below the
    group's largest (7 2^-13 of S) and rounds its FP32 accumulator once per 16 products
    (K / 16 roundings of 2^-24, and as much again for the cut of the smaller addend);
  FP32 output: the bf16 instruction cuts 8 products to 24 bits (8 2^-24) and rounds once per 8;
then alpha, beta and the output conversion: 2^-24 each, and half a step of the output type
(2^-8 bf16, 2^-11 FP16).  Four to eight partial sums of split K add 8 2^-24.
"""
import numpy as np
import pytest

import block_scaled_precision_fp8_amd as bs
from gpu_common import from_dev, guarded, say, to_dev, untouched
from oracle import block128 as ref

pytestmark = pytest.mark.gpu

# half of torch.finfo(t).eps: bf16 keeps 7 fraction bits (eps 2^-7), FP16 10, FP32 23
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def tol(out, K):
    if out == "f32":
        return (8 + 2 * K / 8 + 8 + 2) * 2.0 ** -24 + HALF[out]
    return 7 * 2.0 ** -13 + (2 * K / 16 + 8 + 2) * 2.0 ** -24 + HALF[out]


def values(rows, k, dtype, seed):
    import torch
    g = np.random.default_rng(seed)
    x = g.standard_normal((rows, k)) * np.exp2(g.integers(-12, 6, (rows, 1))) * np.exp2(g.integers(-6, 7, (1, k)))
    x[g.random((rows, k)) < 0.05] = 0
    return torch.from_numpy(x.astype(np.float32)).to(dtype)


# ------------------------------------------------------------------ quantiser
SHAPES = [(1, 1), (1, 128), (3, 40), (16, 512), (128, 128), (129, 127), (130, 257), (64, 1000), (257, 640),
          (1, 8192), (33, 2049), (600, 700), (513, 130), (130, 1300)]


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,k", SHAPES)
def test_quantize(rows, k, block_rows, dtype):
    import torch
    x = values(rows, k, getattr(torch, dtype), rows * 10007 + k)
    xf = x.float().numpy()
    fmt = "e4m3" if (rows + k) % 2 else "e5m2"
    for want in ("rows", "transposed", "both"):
        say(f"quantize_block128 {rows}x{k} {dtype} block_rows={block_rows} {fmt} {want}")
        got = [from_dev(t) for t in bs.fp8_quantize_block128(x.cuda(), fmt, block_rows, rows=want != "transposed",
                                                             transposed=want != "rows")]
        exp = []
        if want != "transposed":
            exp += ref.quantize(xf, fmt, block_rows)
        if want != "rows":
            exp += ref.quantize(np.ascontiguousarray(xf.T), fmt, block_rows)
        assert len(got) == len(exp)
        for a, b in zip(got, exp):
            assert a.shape == b.shape and np.array_equal(a, b)


@pytest.mark.parametrize("off,extra", [(0, 8), (1, 0), (0, 3), (4, 4)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_quantize_strides_offsets_and_guards(dtype, off, extra):
    """Views at odd offsets and row strides, outputs inside canaries."""
    import torch
    rows, k = 70, 200
    x = values(rows, k, getattr(torch, dtype), 5)
    base = torch.zeros(rows * (k + extra) + off + 8, dtype=x.dtype, device="cuda")
    view = base[off:off + rows * (k + extra)].view(rows, k + extra)[:, :k]
    view.copy_(x)
    shapes = [(70, 224), bs.block128_scale_shape(70, 200, 1), (200, 96), bs.block128_scale_shape(200, 70, 1)]
    bufs = [guarded((int(np.prod(s)),), torch.uint8, tail=64) for s in shapes]
    outs = [v.view(s) for (_, v), s in zip(bufs, shapes)]
    say(f"quantize_block128 view offset {off} extra {extra} {dtype}")
    bs.fp8_quantize_block128(view, "e4m3", 1, True, True, *outs)
    xf = x.float().numpy()
    exp = ref.quantize(xf, "e4m3", 1) + ref.quantize(np.ascontiguousarray(xf.T), "e4m3", 1)
    for (buf, _), o, e, s in zip(bufs, outs, exp, shapes):
        assert np.array_equal(from_dev(o), e)
        assert untouched(buf, (int(np.prod(s)),), tail=64)


def test_quantize_special_values():
    import torch
    x = torch.ones(200, 300)
    x[0, 5], x[150, 299], x[3, 200] = float("inf"), float("nan"), -float("inf")
    x[10] = 0.0
    x[11] = -0.0
    x[12] = 2.0 ** -140
    x[13], x[14] = 3.4e38, -1e-38
    for block_rows in (1, 128):
        for fmt in ("e4m3", "e5m2"):
            say(f"quantize_block128 special values block_rows={block_rows} {fmt}")
            got = [from_dev(t) for t in bs.fp8_quantize_block128(x.cuda(), fmt, block_rows, True, True)]
            xf = x.numpy()
            codes, scales = ref.quantize(xf, fmt, block_rows)
            codes_t, scales_t = ref.quantize(np.ascontiguousarray(xf.T), fmt, block_rows)
            for a, b in zip(got, (codes, scales, codes_t, scales_t)):
                assert np.array_equal(a, b)
            rows_only = [from_dev(t) for t in bs.fp8_quantize_block128(x.cuda(), fmt, block_rows)]
            assert np.array_equal(rows_only[0], codes) and np.array_equal(rows_only[1], scales)


# ------------------------------------------------------------------ GEMM
def operand(rows, K, block_rows, fmt, seed):
    g = np.random.default_rng(seed)
    top = 0x7F if fmt == "e4m3" else 0x7C
    codes = g.integers(0, top, (rows, K), dtype=np.uint8) | (g.integers(0, 2, (rows, K), dtype=np.uint8) << 7)
    shape = bs.block128_scale_shape(rows, K, block_rows)
    return codes, g.integers(115, 133, shape, dtype=np.uint8)


def check(d, d_ref, s_ref, out, K, alpha=1.0, beta=0.0, c=0.0, label=""):
    r = alpha * d_ref + beta * np.asarray(c, dtype=np.float64)
    bound = abs(alpha) * s_ref + np.abs(beta * np.asarray(c, dtype=np.float64))
    err = np.abs(np.asarray(d, dtype=np.float64) - r)
    # FP16 results below its normal range are rounded to 2^-25
    over = err - (2.0 ** -25 if out == "f16" else 0.0) - tol(out, K) * bound
    say(f"{label}: worst error / S {float((err / np.maximum(bound, 1e-300)).max()):.3e}, tolerance {tol(out, K):.3e}")
    assert np.all(over <= 0), f"{label}: {over.max()}"


def run_gemm(M, N, K, a_rows, b_rows, a_fmt, b_fmt, out, seed=0, alpha=1.0, beta=0.0, extra=0):
    import torch
    a, sa = operand(M, K, a_rows, a_fmt, seed)
    b, sb = operand(N, K, b_rows, b_fmt, seed + 1)
    if out == "f16":
        # keep |D| below 65504: the largest values here are 2^8 2^8 (E4M3) or 2^15 (E5M2) times the scales
        sa, sb = sa - (20 if a_fmt == "e4m3" else 27), sb - (0 if b_fmt == "e4m3" else 7)
    dt = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[out]
    buf, d = guarded((M, N), dt, extra_cols=extra, extra_rows=2, tail=32)
    c = None
    if beta:
        d.copy_(torch.from_numpy(np.random.default_rng(seed + 2).standard_normal((M, N))).to(dt))
        c = d.clone()
    label = f"gemm_block128 {M}x{N}x{K} rows {a_rows},{b_rows} {a_fmt}x{b_fmt} {out} alpha {alpha} beta {beta}"
    say(label)
    got = bs.scaled_gemm_block128(to_dev(a), to_dev(sa), to_dev(b), to_dev(sb), a_fmt, b_fmt, a_rows, b_rows, out,
                                  alpha, d if beta else None, beta, d)
    assert got is d
    if M * N * K < 1 << 30:
        d_ref, s_ref = ref.gemm(a, sa, a_fmt, a_rows, b, sb, b_fmt, b_rows)
    else:       # the same product in float64 on the device
        x, y = (to_dev(ref.dequantize(*o)) for o in ((a, sa, a_fmt, a_rows), (b, sb, b_fmt, b_rows)))
        d_ref, s_ref = from_dev(x @ y.t().contiguous()), from_dev(x.abs() @ y.abs().t().contiguous())
    check(from_dev(d), d_ref, s_ref, out, K, alpha, beta, 0.0 if c is None else from_dev(c), label)
    assert untouched(buf, (M, N), extra_cols=extra, extra_rows=2, tail=32)


@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 32), (1, 40, 4096), (16, 300, 160), (33, 65, 96), (17, 128, 544),
                                   (64, 130, 128), (128, 128, 640), (130, 257, 1184), (257, 129, 512)])
def test_gemm_shapes(M, N, K, out):
    run_gemm(M, N, K, 1, 128, "e4m3", "e4m3", out, seed=M + N + K)


@pytest.mark.parametrize("a_rows", [1, 128])
@pytest.mark.parametrize("b_rows", [1, 128])
@pytest.mark.parametrize("a_fmt,b_fmt", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_gemm_blocks_and_formats(a_rows, b_rows, a_fmt, b_fmt, out):
    run_gemm(150, 200, 672, a_rows, b_rows, a_fmt, b_fmt, out, seed=3)


@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("alpha,beta,extra", [(0.5, 0.0, 8), (1.0, 1.0, 0), (2.0, -0.5, 3)])
@pytest.mark.parametrize("M,N,K", [(20, 70, 256), (300, 260, 160)])
def test_gemm_epilogue(M, N, K, alpha, beta, extra, out):
    run_gemm(M, N, K, 1, 1, "e5m2", "e4m3", out, seed=9, alpha=alpha, beta=beta, extra=extra)


# shapes at which every form of the kernel runs: 16 rows; 32 x 32 with K split; 128 x 128; 192 x 128; 256 x 128;
# 256 x 256 (several tiles per workgroup), whole and ragged rows of D, an odd and an even number of K blocks
@pytest.mark.parametrize("out", ["bf16", "f32", "f16"])
@pytest.mark.parametrize("M,N,K,a_rows,b_rows,beta", [
    (16, 4096, 2048, 1, 128, 0.0), (9, 1001, 9056, 1, 128, 1.0), (16, 6000, 2048, 1, 1, 0.0), (513, 1030, 1056, 1, 128, 0.0), (1000, 2000, 544, 1, 1, 0.0),
    (2100, 4300, 160, 1, 128, 1.0), (4096, 3500, 288, 128, 1, 0.0), (1111, 4000, 2080, 1, 128, 0.0),
    (1111, 4000, 2080, 1, 1, 1.0), (1500, 5000, 1312, 1, 128, 0.0), (2050, 7003, 3232, 1, 128, 0.0),
    (3900, 4000, 3232, 128, 128, 0.0), (3900, 4000, 3232, 1, 1, 1.0), (5000, 9000, 4128, 1, 128, 0.0)])
def test_gemm_forms(M, N, K, a_rows, b_rows, beta, out):
    run_gemm(M, N, K, a_rows, b_rows, "e4m3", "e4m3", out, seed=K, beta=beta)


def test_gemm_is_reproducible_and_rows_do_not_depend_on_others():
    """The same call twice gives the same bits; a row's result is the same alone and among others as long
    as the same form runs."""
    a, sa = operand(2100, 672, 1, "e4m3", 5)
    b, sb = operand(4300, 672, 128, "e4m3", 6)
    t = [to_dev(x) for x in (a, sa, b, sb)]
    say("gemm_block128 twice")
    d = bs.scaled_gemm_block128(*t)
    for _ in range(3):
        assert np.array_equal(from_dev(bs.scaled_gemm_block128(*t)), from_dev(d))


def test_gemm_empty_and_k_zero():
    import torch
    z = torch.zeros((0, 64), dtype=torch.uint8, device="cuda")
    b, sb = operand(40, 64, 128, "e4m3", 1)
    say("gemm_block128 empty")
    s0 = torch.zeros(bs.block128_scale_shape(0, 64, 1), dtype=torch.uint8, device="cuda")
    assert bs.scaled_gemm_block128(z, s0, to_dev(b), to_dev(sb)).shape == (0, 40)
    e = torch.zeros((3, 0), dtype=torch.uint8, device="cuda")
    f = torch.zeros((5, 0), dtype=torch.uint8, device="cuda")
    s = [torch.zeros(bs.block128_scale_shape(r, 0, n), dtype=torch.uint8, device="cuda") for r, n in ((3, 1), (5, 128))]
    d = torch.full((3, 5), 2.0, device="cuda")
    assert not from_dev(bs.scaled_gemm_block128(e, s[0], f, s[1], out="f32")).any()
    bs.scaled_gemm_block128(e, s[0], f, s[1], out="f32", c=d, beta=0.5, d=d)
    assert np.all(from_dev(d) == 1.0)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(16, 64, 512), (200, 300, 512), (2100, 4300, 320)])
def test_gemm_nan_scale_and_unused_scale_bytes(M, N, K, out):
    """A NaN scale makes its row NaN and no other; the unused bytes of the last word do not matter."""
    import torch
    for k in (K, K - 160):
        a, sa = operand(M, k, 1, "e4m3", 1)
        b, sb = operand(N, k, 128, "e4m3", 2)
        nkb = (k + 127) // 128
        if nkb % 4:
            sa[-1, :, nkb % 4:] = 255
            sb[-1, :, nkb % 4:] = 255
        sa[0, 7, 1] = 255
        say(f"gemm_block128 NaN scale {M}x{N}x{k} {out}")
        d = from_dev(bs.scaled_gemm_block128(to_dev(a), to_dev(sa), to_dev(b), to_dev(sb), out=out))
        d_ref, s_ref = ref.gemm(a, sa, "e4m3", 1, b, sb, "e4m3", 128)
        assert np.isnan(d[7]).all()
        keep = np.arange(M) != 7
        check(d[keep], d_ref[keep], s_ref[keep], out, k, label="other rows")


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(5, 40, 700), (64, 100, 300), (300, 300, 1000), (2100, 4300, 300)])
def test_gemm_carries_non_finite_inputs(M, N, K, out):
    """An infinity in x makes its row of x w^T NaN and leaves the others; NaN codes do the same."""
    import torch
    x, w = values(M, K, torch.float32, 1), values(N, K, torch.float32, 2)
    x[M // 2, 200] = float("inf")
    say(f"gemm_block128 non-finite {M}x{N}x{K} {out}")
    xq, xs = bs.fp8_quantize_block128(x.cuda(), "e4m3", 1)
    wq, ws = bs.fp8_quantize_block128(w.cuda(), "e4m3", 128)
    d = from_dev(bs.scaled_gemm_block128(xq, xs, wq, ws, out=out))
    keep = np.arange(M) != M // 2
    assert np.isnan(d[M // 2]).all() and np.isfinite(d[keep]).all()
    xs.clamp_(max=200)          # the scale byte no longer says NaN: the codes still do
    d = from_dev(bs.scaled_gemm_block128(xq, xs, wq, ws, out=out))
    assert np.isnan(d[M // 2]).all() and np.isfinite(d[keep]).all()


@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [(7, 120, 256), (50, 120, 256), (300, 264, 256), (2100, 4304, 160)])
def test_gemm_output_at_an_odd_address(M, N, K, out):
    """D one element into a buffer, with an odd row stride: no 16-byte stores."""
    import torch
    a, sa = operand(M, K, 1, "e4m3", 5)
    b, sb = operand(N, K, 128, "e4m3", 6)
    if out == "f16":
        sa = sa - 20
    dt = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[out]
    buf, view = guarded((M, N + 1), dt, extra_cols=2, extra_rows=1, tail=16)
    before = buf.clone()
    say(f"gemm_block128 odd address {M}x{N}x{K} {out}")
    t = [to_dev(v) for v in (a, sa, b, sb)]
    bs.scaled_gemm_block128(*t, out=out, d=view[:, 1:])
    assert torch.equal(view[:, 1:], bs.scaled_gemm_block128(*t, out=out))
    view[:, 1:] = 0
    grid, want = buf.view(torch.uint8), before
    want[: M * (N + 3)].view(M, N + 3)[:, 1:N + 1] = 0
    assert torch.equal(grid, want.view(torch.uint8))


def test_gemm_extreme_scales():
    """Scale bytes at both ends: products are FP32 values as long as they are normal there."""
    import torch
    a, sa = operand(40, 256, 1, "e4m3", 1)
    b, sb = operand(50, 256, 1, "e4m3", 2)
    for pa, pb in ((0, 230), (235, 20), (20, 235), (127, 127)):
        sa[:], sb[:] = pa, pb
        for out in ("f32", "bf16"):
            say(f"gemm_block128 scales {pa},{pb} {out}")
            d = from_dev(bs.scaled_gemm_block128(to_dev(a), to_dev(sa), to_dev(b), to_dev(sb), b_block_rows=1, out=out))
            d_ref, s_ref = ref.gemm(a, sa, "e4m3", 1, b, sb, "e4m3", 1)
            if out == "f32" and pa == 0:
                continue    # 2^-127 times a code is below bf16's normal range: covered by the 16-bit outputs
            check(d, d_ref, s_ref, out, 256, label="extreme")


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("M,N,K", [(9, 50, 256), (40, 50, 256), (300, 264, 544), (2100, 4304, 160)])
def test_gemm_smallest_scale(M, N, K, fmt, out):
    """Scale byte 0 (2^-127) on either side, codes of 2 and more: dequantised magnitudes are 2^-126 and more."""
    a, sa = operand(M, K, 1, fmt, 1)
    b, sb = operand(N, K, 128, fmt, 2)
    two = 0x40
    a, b = a | two, b | two
    for pa, pb in ((0, 230), (230, 0)):
        # E4M3: | 0x40 could make the NaN code 0x7F
        x, y = (np.where((t & 0x7F) >= (0x7F if fmt == "e4m3" else 0x7C), 0x41, t).astype(np.uint8) for t in (a, b))
        sa[:], sb[:] = pa, pb
        label = f"gemm_block128 {M}x{N}x{K} {fmt} scales {pa},{pb} {out}"
        say(label)
        d = bs.scaled_gemm_block128(to_dev(x), to_dev(sa), to_dev(y), to_dev(sb), fmt, fmt, 1, 128, out)
        u, v = to_dev(ref.dequantize(x, sa, fmt, 1)), to_dev(ref.dequantize(y, sb, fmt, 128))
        d_ref, s_ref = from_dev(u @ v.t().contiguous()), from_dev(u.abs() @ v.abs().t().contiguous())
        check(from_dev(d), d_ref, s_ref, out, K, label=label)


# ------------------------------------------------------------------ a linear layer's three products
def test_layer_products_from_quantised_operands():
    """y = x w^T, dx = g w, dw = g^T x from the quantiser's outputs, against float64 products of the
    dequantised operands and, loosely, of the originals."""
    import torch
    T, O, I = 150, 200, 330
    x, w, g = (values(*s, torch.bfloat16, i) for i, s in enumerate(((T, I), (O, I), (T, O))))
    x, w, g = x / x.abs().max(), w.float() / w.abs().max(), g / g.abs().max()
    say("layer products")
    xq, xs, xqt, xst = bs.fp8_quantize_block128(x.cuda(), "e4m3", 1, True, True)
    wq, ws, wqt, wst = bs.fp8_quantize_block128(w.float().cuda(), "e4m3", 128, True, True)
    gq, gs, gqt, gst = bs.fp8_quantize_block128(g.cuda(), "e5m2", 1, True, True)
    y = bs.scaled_gemm_block128(xq, xs, wq, ws, out="f32")
    dx = bs.scaled_gemm_block128(gq, gs, wqt, wst, "e5m2", "e4m3", out="f32")
    dw = torch.zeros((O, I), device="cuda")
    for _ in range(2):
        bs.scaled_gemm_block128(gqt, gst, xqt, xst, "e5m2", "e4m3", 1, 1, out="f32", c=dw, beta=1.0, d=dw)
    xf, wf, gf = (t.double().numpy() for t in (x, w, g))
    # relative rounding of codes: 2^-4 (E4M3), 2^-3 (E5M2); codes below the normal range lose at most half
    # their step, 2^-10 / 448 (2^-17 / 57344) of twice the block's maximum, here 1
    ea, eg = 2.0 ** -4, 2.0 ** -3
    for got, p, q, ep, eq, n in ((y, xf, wf.T, ea, ea, I), (dx, gf, wf, eg, ea, O), (dw, 2 * gf.T, xf, eg, ea, T)):
        err = np.abs(from_dev(got) - p @ q)
        rel = ((1 + ep) * (1 + eq) - 1) * (np.abs(p) @ np.abs(q))
        assert np.all(err <= rel * 1.001 + n * 2 * 2.0 ** -17)


# ------------------------------------------------------------------ streams and graphs
def test_two_streams_at_once():
    """Independent calls on two streams, no shared state between them."""
    import torch
    say("block128 on two streams")
    w, ws = bs.fp8_quantize_block128(values(3000, 2048, torch.float32, 1).cuda(), "e4m3", 128)
    xs = [values(m, 2048, torch.bfloat16, m).cuda() for m in (16, 700, 1800, 2100)]
    want = [bs.scaled_gemm_block128(*bs.fp8_quantize_block128(x), w, ws) for x in xs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for i in range(24):
        with torch.cuda.stream(streams[i % 2]):
            got.append(bs.scaled_gemm_block128(*bs.fp8_quantize_block128(xs[i % 4]), w, ws))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i % 4]) for i, g in enumerate(got))


def test_stream_and_graph():
    import torch
    M, N, K = 48, 300, 400
    x, w = values(M, K, torch.bfloat16, 1).cuda(), values(N, K, torch.float32, 2).cuda()
    wq, ws = bs.fp8_quantize_block128(w, "e4m3", 128)
    xq, xs = bs.fp8_quantize_block128(x, "e4m3", 1)
    want = bs.scaled_gemm_block128(xq, xs, wq, ws)
    torch.cuda.synchronize()
    say("block128 on a side stream")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a = bs.fp8_quantize_block128(x, "e4m3", 1)
        d = bs.scaled_gemm_block128(*a, wq, ws)
    side.synchronize()
    assert torch.equal(d, want)
    say("block128 in a graph")
    graph = torch.cuda.CUDAGraph()
    out = torch.empty_like(want)
    with torch.cuda.graph(graph):
        a = bs.fp8_quantize_block128(x, "e4m3", 1)
        bs.scaled_gemm_block128(*a, wq, ws, d=out)
    for i in range(4):
        x.copy_(values(M, K, torch.bfloat16, 10 + i))
        graph.replay()
        torch.cuda.synchronize()
        eager = bs.scaled_gemm_block128(*bs.fp8_quantize_block128(x, "e4m3", 1), wq, ws)
        assert torch.equal(out, eager)


def test_writes_count_in_autograd_versions():
    """A graph that saved a tensor which a call then writes refuses to use the new values."""
    import torch
    x = values(40, 96, torch.float32, 1).cuda()
    q, s = bs.fp8_quantize_block128(x)
    w = torch.ones(40, 40, device="cuda", requires_grad=True)
    for beta in (0.0, 1.0):
        d = torch.ones(40, 40, device="cuda")
        y = (w * d).sum()
        say(f"gemm_block128 into a saved tensor, beta {beta}")
        bs.scaled_gemm_block128(q, s, q, s, b_block_rows=1, out="f32", c=d, beta=beta, d=d)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()
    say("quantize_block128 into given outputs")
    outs = bs.fp8_quantize_block128(x, "e4m3", 1, True, True)
    before = [t._version for t in outs]
    bs.fp8_quantize_block128(x, "e4m3", 1, True, True, *outs)
    assert [t._version for t in outs] == [n + 1 for n in before]
    with torch.inference_mode():
        d = torch.zeros(40, 40, device="cuda")      # counts no versions
    bs.scaled_gemm_block128(q, s, q, s, b_block_rows=1, out="f32", d=d)
    assert from_dev(d).any()


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_quantize_padding_codes(fmt, block_rows):
    """Columns k .. kp - 1: zeros, but NaN codes in a block with a non-finite value."""
    import torch
    x = torch.ones(130, 140)
    x[1, 139] = float("inf")
    say(f"quantize_block128 padding block_rows={block_rows} {fmt}")
    for transposed in (False, True):
        y = x.t().contiguous() if transposed else x
        codes = from_dev(bs.fp8_quantize_block128(y.cuda(), fmt, block_rows, not transposed, transposed)[0])
        bad = np.arange(130) // block_rows == 1 // block_rows
        assert codes.shape == (130, 160) and np.all(codes[bad, 128:] == 0x7F) and not codes[~bad, 140:].any()
