"""The block-of-128 GEMM in each of its kernel forms, and with several tiles per workgroup where the
form is persistent (MI355X): outputs and epilogues, format pairs, special scale bytes, odd addresses,
repeated calls, rows alone and among others.

Every case asserts the form that its shape takes (tests/block128_forms.py).  References are float64
products on the device; tolerances are those of test_gpu_block128.py.  Its 8 2^-24 for partial sums
covers the up to 16 of the rows form too: with w waves each of them adds at most 128 ceil(K / (512 w))
roundings of its own and the join w - 1, together below the 2 K / 8 + 8 that one chain is given.
"""
import numpy as np
import pytest

import block_scaled_precision_fp8_amd as bs
from block128_forms import form
from gpu_common import from_dev, guarded, say, to_dev, untouched
from oracle import block128 as ref
from test_gpu_block128 import operand, tol

# (M, N, K) by form and tiles per workgroup; N a multiple of 8.  K: an even and an odd number of K
# blocks, loops that end on a whole and on half a group of four, a partial last block.
SIXTEEN = {
    ("rows", 1): [(9, 1000, 9056), (16, 4096, 2048)],
    ("32x32", 1): [(48, 1000, 672), (200, 520, 1280)],
    ("128x128", 1): [(200, 7176, 192), (760, 1584, 576)],
    ("192x128", 1): [(444, 8336, 480), (1111, 4000, 2080)],
    ("192x128", 2): [(1297, 8912, 480), (1300, 8912, 768), (1297, 8912, 576)],
    ("192x128", 4): [(1700, 14336, 1024)],
    ("256x128", 1): [(627, 8336, 1248)],
    ("256x128", 2): [(1588, 7560, 1248), (1588, 7560, 1536), (1600, 7560, 1344)],
    ("256x128", 5): [(2696, 13400, 1248)],
    ("256x256", 2): [(3916, 7752, 3232), (3916, 7752, 3584)],
}
FP32 = {
    ("rows", 1): SIXTEEN["rows", 1],
    ("32x32", 1): SIXTEEN["32x32", 1],
    ("128x128", 1): [(200, 7752, 384), (1300, 1584, 192)],
    ("192x128", 1): [(444, 8336, 480)],
    ("192x128", 2): [(1297, 8912, 480), (1300, 8912, 768), (1297, 8912, 576)],
    ("256x256", 1): [(1588, 7560, 1248)],
    ("256x256", 2): [(3722, 7560, 1248), (3722, 7560, 1536), (3722, 7560, 1344)],
}
DTYPES = {"f32": "float32", "bf16": "bfloat16", "f16": "float16"}


def cases(first=False, outs=("bf16", "f16", "f32")):
    """(form, tiles, M, N, K, out) for the given outputs; first: one shape per form."""
    return [(*key, *s, out) for out in outs for key, shapes in (FP32 if out == "f32" else SIXTEEN).items()
            for s in (shapes[:1] if first else shapes)]


@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_shapes_take_the_forms_they_name(out):
    for name, tiles, M, N, K, _ in cases(outs=(out,)):
        assert form(M, N, K, out) == (name, tiles), (M, N, K)
        assert form(M, N - 3, K, out) == (name, tiles), (M, N - 3, K)


def inputs(M, N, K, a_rows, b_rows, a_fmt, b_fmt, out, seed):
    a, sa = operand(M, K, a_rows, a_fmt, seed)
    b, sb = operand(N, K, b_rows, b_fmt, seed + 1)
    if out == "f16":        # keep |D| below 65504
        sa, sb = sa - (20 if a_fmt == "e4m3" else 27), sb - (0 if b_fmt == "e4m3" else 7)
    return a, sa, b, sb


def products(a, sa, a_fmt, a_rows, b, sb, b_fmt, b_rows):
    """(D, S) in float64, on the device."""
    x, y = to_dev(ref.dequantize(a, sa, a_fmt, a_rows)), to_dev(ref.dequantize(b, sb, b_fmt, b_rows)).t().contiguous()
    return x @ y, x.abs() @ y.abs()


def check(d, d_ref, s_ref, out, K, label):
    err = (d.double() - d_ref).abs()
    # FP16 results below its normal range are rounded to 2^-25
    over = err - (2.0 ** -25 if out == "f16" else 0.0) - tol(out, K) * s_ref
    say(f"{label}: worst error / S {float((err / s_ref.clamp(min=1e-300)).max()):.3e}, tolerance {tol(out, K):.3e}")
    assert bool((over <= 0).all()), f"{label}: {float(over.max())}"     # NaN fails too


def run(name, tiles, M, N, K, out, a_rows=1, b_rows=128, a_fmt="e4m3", b_fmt="e4m3", alpha=1.0, beta=0.0, seed=0):
    import torch
    assert form(M, N, K, out) == (name, tiles)
    t = inputs(M, N, K, a_rows, b_rows, a_fmt, b_fmt, out, seed)
    a, sa, b, sb = t
    buf, d = guarded((M, N), getattr(torch, DTYPES[out]), extra_cols=8, extra_rows=2, tail=32)
    if beta:
        d.normal_()
    c = d.double() if beta else None
    label = f"gemm_block128 {name} x{tiles} {M}x{N}x{K} rows {a_rows},{b_rows} {a_fmt}x{b_fmt} {out} alpha {alpha} beta {beta}"
    say(label)
    bs.scaled_gemm_block128(*map(to_dev, t), a_fmt, b_fmt, a_rows, b_rows, out, alpha, d if beta else None, beta, d)
    d_ref, s_ref = products(a, sa, a_fmt, a_rows, b, sb, b_fmt, b_rows)
    d_ref, s_ref = alpha * d_ref, abs(alpha) * s_ref
    if beta:
        d_ref, s_ref = d_ref + beta * c, s_ref + (beta * c).abs()
    check(d, d_ref, s_ref, out, K, label)
    assert untouched(buf, (M, N), extra_cols=8, extra_rows=2, tail=32)


@pytest.mark.gpu
@pytest.mark.parametrize("name,tiles,M,N,K,out", cases())
def test_whole_columns(name, tiles, M, N, K, out):
    """Without C: bf16 leaves by constant-count stores, which may be in flight into the next tile."""
    run(name, tiles, M, N, K, out, seed=K)


@pytest.mark.gpu
@pytest.mark.parametrize("name,tiles,M,N,K,out", cases())
def test_ragged_columns_and_c(name, tiles, M, N, K, out):
    run(name, tiles, M, N - 3, K, out, alpha=0.5, beta=-1.0, seed=K + 1)


@pytest.mark.gpu
@pytest.mark.parametrize("a_fmt,b_fmt", [("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("name,tiles,M,N,K,out", cases(True, ("bf16", "f32")))
def test_format_pairs(name, tiles, M, N, K, out, a_fmt, b_fmt):
    """As dx = g w and dW = g^T x have them, blocks of 1 x 128 and 128 x 128 on either side."""
    run(name, tiles, M, N, K, out, *((1, 1) if a_fmt == b_fmt else (128, 1) if a_fmt == "e4m3" else (1, 128)), a_fmt, b_fmt,
        seed=K + 2)


@pytest.mark.gpu
@pytest.mark.parametrize("name,tiles,M,N,K,out", cases(True, ("bf16", "f32")))
def test_nan_scale_and_unused_scale_bytes(name, tiles, M, N, K, out):
    """A NaN scale makes its row NaN and no other; the unused bytes of the last word do not matter."""
    a, sa, b, sb = inputs(M, N, K, 1, 128, "e4m3", "e4m3", out, 1)
    used = (K + 127) // 128 % 4
    row, kb = M - 2, K // 128
    clean = sa.copy()
    if used:
        sa[-1, :, used:] = sb[-1, :, used:] = 255
    sa[kb // 4 if kb * 128 < K else 0, row, kb % 4 if kb * 128 < K else 1] = 255
    say(f"gemm_block128 {name} x{tiles} NaN scale {M}x{N}x{K} {out}")
    d = bs.scaled_gemm_block128(*map(to_dev, (a, sa, b, sb)), out=out)
    d_ref, s_ref = products(a, clean, "e4m3", 1, b, sb, "e4m3", 128)
    assert bool(d[row].isnan().all())
    d[row], d_ref[row] = 0, 0
    check(d, d_ref, s_ref, out, K, "other rows")


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("name,tiles,M,N,K,out", cases(True, ("bf16", "f32")))
def test_ends_of_the_scales(name, tiles, M, N, K, out, fmt):
    """The smallest scale byte, with codes of 2 and more (magnitudes of 2^-126 and more), and the largest
    at which every code is below 2^128, each against a moderate one on the other side."""
    a, sa, b, sb = inputs(M, N, K, 1, 128, fmt, fmt, out, 3)
    two = [t | 0x40 for t in (a, b)]
    two = [np.where((t & 0x7F) >= (0x7F if fmt == "e4m3" else 0x7C), 0x41, t).astype(np.uint8) for t in two]
    top = 246 if fmt == "e4m3" else 239
    for (x, y), pa, pb in ((two, 0, 230), (two, 230, 0), ((a, b), top, 20), ((a, b), 20, top)):
        sa[:], sb[:] = pa, pb
        label = f"gemm_block128 {name} x{tiles} {M}x{N}x{K} {fmt} scales {pa},{pb} {out}"
        say(label)
        d = bs.scaled_gemm_block128(*map(to_dev, (x, sa, y, sb)), fmt, fmt, out=out)
        check(d, *products(x, sa, fmt, 1, y, sb, fmt, 128), out, K, label)


@pytest.mark.gpu
@pytest.mark.parametrize("name,tiles,M,N,K", [c[:5] for c in cases(True, ("bf16",))])
def test_magnitudes_beyond_fp32(name, tiles, M, N, K):
    """Dequantised magnitudes of 2^128 and more, as the quantiser writes them for values next to FP32's
    largest: 16-bit outputs multiply them out, FP32 output counts them as infinite."""
    import torch
    x, w = torch.ones(M, K, device="cuda"), torch.full((N, K), 2.0 ** -100, device="cuda")
    x[M - 1] = 3.4e38
    say(f"gemm_block128 {name} x{tiles} {M}x{N}x{K} beyond FP32")
    t = bs.fp8_quantize_block128(x) + bs.fp8_quantize_block128(w, block_rows=128)
    d = bs.scaled_gemm_block128(*t)
    # 256 2^120 2^-100 K: bf16 rounds K 2^28 by at most half a step, the sum by tol
    assert bool(((d[M - 1].double() / (K * 2.0 ** 28) - 1).abs() <= tol("bf16", K)).all())
    d = bs.scaled_gemm_block128(*t, out="f32")
    assert not bool(d[M - 1].isfinite().any()) and bool(d[:M - 1].isfinite().all())


@pytest.mark.gpu
@pytest.mark.parametrize("name,tiles,M,N,K,out", cases(True))
def test_odd_addresses(name, tiles, M, N, K, out):
    """D one element into a buffer, with an odd row stride: no 16-byte stores; the same bits."""
    import torch
    t = [to_dev(v) for v in inputs(M, N, K, 1, 128, "e4m3", "e4m3", out, 5)]
    buf, view = guarded((M, N + 1), getattr(torch, DTYPES[out]), extra_cols=2, extra_rows=1, tail=16)
    want = buf.clone()
    say(f"gemm_block128 {name} x{tiles} odd address {M}x{N}x{K} {out}")
    bs.scaled_gemm_block128(*t, out=out, d=view[:, 1:])
    assert torch.equal(view[:, 1:], bs.scaled_gemm_block128(*t, out=out))
    for b in (buf, want):
        b[: M * (N + 3)].view(M, N + 3)[:, 1:N + 1] = 0
    assert torch.equal(buf.view(torch.uint8), want.view(torch.uint8))


@pytest.mark.gpu
@pytest.mark.parametrize("name,tiles,M,N,K,out", cases(True))
def test_repeated_calls_and_rows_alone(name, tiles, M, N, K, out):
    """The same call gives the same bits; so do some of its rows and columns alone, where they take the
    same form (the order of a sum is the form's, not the place's in the matrix)."""
    import torch
    t = [to_dev(v) for v in inputs(M, N, K, 1, 128, "e4m3", "e4m3", out, 6)]
    a, sa, b, sb = t
    say(f"gemm_block128 {name} x{tiles} repeated {M}x{N}x{K} {out}")
    d = bs.scaled_gemm_block128(*t, out=out)
    for _ in range(3):
        assert torch.equal(bs.scaled_gemm_block128(*t, out=out), d)
    parts = 0
    for m0, n0 in ((7, 0), (1, 128), (0, 256), (M // 64, 128)):
        if form(M - m0, N - n0, K, out)[0] != name:
            continue
        parts += 1
        say(f"gemm_block128 {name} rows from {m0}, columns from {n0}")
        got = bs.scaled_gemm_block128(a[m0:].contiguous(), sa[:, m0:].contiguous(), b[n0:].contiguous(),
                                      sb[:, n0 // 128:].contiguous(), out=out)
        assert torch.equal(got, d[m0:, n0:])
    assert parts
