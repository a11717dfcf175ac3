"""Refusals of the norm and of the grouped entry points, from the host's checks (CPU): every call here
returns before anything could be launched."""
import pytest

import block_scaled_precision_fp8_amd as bs

OK, INVALID, UNSUPPORTED = 0, 1, 2
E4M3, E5M2, MXFP4 = 0, 1, 2
F32, BF16, F16 = 0, 1, 2
P = 0x10000


@pytest.fixture(scope="module")
def L():
    return bs.lib()


def caller(fn, names, good):
    def call(**kw):
        return fn(*[{**good, **kw}[n] for n in names.split()])
    return call


def test_norm(L):
    call = caller(L.rmsnorm_quantize_block128,
                  "x x_type rows k ldx residual h_type ldr weight w_type eps fmt codes scales y y_type ldy h ldh rstd stream",
                  dict(x=P, x_type=BF16, rows=0, k=64, ldx=64, residual=P, h_type=BF16, ldr=64, weight=P, w_type=F32,
                       eps=1e-6, fmt=E4M3, codes=P, scales=P, y=P, y_type=F32, ldy=64, h=P, ldh=64, rstd=P, stream=None))
    assert call() == OK and call(rows=4, k=0) == OK
    assert call(fmt=MXFP4) == UNSUPPORTED
    for t in ("x_type", "h_type", "w_type", "y_type"):
        assert call(**{t: 3}) == UNSUPPORTED
    r = dict(rows=4)
    assert call(**r, k=32769, ldx=32769, ldr=32769, ldh=32769, ldy=32769) == UNSUPPORTED
    assert call(rows=-1) == INVALID and call(**r, k=-1) == INVALID and call(rows=1 << 31) == INVALID
    for eps in (-1.0, float("nan"), float("inf")):
        assert call(eps=eps) == INVALID
    for ld in ("ldx", "ldr", "ldh", "ldy"):
        assert call(**r, **{ld: 63}) == INVALID
    assert call(**r, codes=0) == INVALID and call(**r, scales=0) == INVALID
    assert call(**r, codes=0, scales=0, y=0) == INVALID         # nothing to write
    assert call(**r, residual=0) == INVALID and call(**r, h=0) == INVALID and call(**r, x=0) == INVALID
    for p, off in (("x", 1), ("residual", 1), ("h", 1), ("weight", 2), ("y", 2), ("rstd", 2), ("codes", 8), ("scales", 2)):
        assert call(**r, **{p: P + off}) == INVALID, p


def test_norm_backward(L):
    call = caller(L.rmsnorm_backward,
                  "dy dy_type ldy h h_type ldh rstd weight w_type dh dh_type lddh rows k dx ldx dweight accumulate "
                  "workspace size stream",
                  dict(dy=P, dy_type=BF16, ldy=64, h=P, h_type=BF16, ldh=64, rstd=P, weight=P, w_type=BF16, dh=P,
                       dh_type=F32, lddh=64, rows=4, k=0, dx=P, ldx=64, dweight=P, accumulate=0, workspace=P,
                       size=1 << 30, stream=None))
    assert call() == OK
    for t in ("dy_type", "h_type", "w_type", "dh_type"):
        assert call(**{t: 3}) == UNSUPPORTED
    k = dict(k=64)
    assert call(k=32769) == UNSUPPORTED
    assert call(rows=-1) == INVALID and call(k=-1) == INVALID and call(rows=1 << 31) == INVALID
    assert call(accumulate=2) == INVALID
    for p in ("dy", "h", "rstd", "dx", "workspace"):
        assert call(**k, **{p: 0}) == INVALID, p
    for ld in ("ldy", "ldh", "lddh", "ldx"):
        assert call(**k, **{ld: 63}) == INVALID, ld
    for p, off in (("dy", 1), ("h", 1), ("dx", 1), ("rstd", 2), ("weight", 1), ("dh", 2), ("dweight", 2), ("workspace", 8)):
        assert call(**k, **{p: P + off}) == INVALID, p
    need = L.rmsnorm_backward_workspace(4, 64)
    assert need >= 64 * 4 and call(**k, size=need - 1) == INVALID
    for bad in ((-1, 4), (4, -1), (0, 4), (4, 0), (1 << 31, 4), (4, 32769)):
        assert L.rmsnorm_backward_workspace(*bad) == 0


def test_shapes(L):
    assert L.block128_grouped_columns(0, 8) == L.block128_grouped_words(0, 8) == 0
    for rows in (1, 2, 127, 128, 129, 1000, 1 << 30):
        for groups in (1, 2, 3, 64, 1024):
            n = min(rows, groups)
            # the most columns: n - 1 groups of one row, the rest in the last; the most words likewise
            worst = (n - 1) * 128 + (rows - n + 1 + 127) // 128 * 128
            assert L.block128_grouped_columns(rows, groups) >= worst and L.block128_grouped_columns(rows, groups) % 128 == 0
            assert L.block128_grouped_words(rows, groups) >= n - 1 + (rows - n + 1 + 511) // 512
    assert L.block128_grouped_columns((1 << 30) + 1, 1) == 0 and L.block128_grouped_columns(4, 1025) == 0
    assert bs.block128_grouped_shape(5, 7, 2) == ((7, 256), (2, 7, 4))


def test_quantize(L):
    call = caller(L.fp8_quantize_grouped_block128,
                  "x x_type source k ld index rows offsets groups fmt codes scales codes_t columns scales_t words stream",
                  dict(x=P, x_type=BF16, source=4, k=64, ld=64, index=0, rows=0, offsets=P, groups=2, fmt=E4M3, codes=P,
                       scales=P, codes_t=P, columns=256, scales_t=P, words=2, stream=None))
    assert call() == OK and call(rows=4, k=0, ld=0) == OK and call(rows=4, groups=0) == OK
    assert call(fmt=MXFP4) == UNSUPPORTED and call(x_type=3) == UNSUPPORTED
    assert call(groups=1025) == UNSUPPORTED and call(rows=(1 << 30) + 1) == UNSUPPORTED
    assert call(rows=-1) == INVALID and call(source=-1) == INVALID and call(groups=-1) == INVALID and call(ld=63) == INVALID
    r = dict(rows=4)
    for p in ("x", "offsets", "codes", "scales", "codes_t", "scales_t"):
        assert call(**r, **{p: 0}) == INVALID, p
    assert call(**r, codes=0, scales=0, codes_t=0, scales_t=0) == INVALID
    assert call(**r, source=3) == INVALID                        # fewer rows than are sorted, without an index
    assert call(**r, columns=128) == INVALID and call(**r, columns=300) == INVALID and call(**r, words=1) == INVALID
    assert call(**r, columns=1 << 31) == INVALID and call(**r, words=1 << 31) == INVALID
    for p, off in (("x", 1), ("index", 2), ("offsets", 2), ("codes", 8), ("codes_t", 8), ("scales", 2), ("scales_t", 2)):
        assert call(**r, **{p: P + off}) == INVALID, p
    assert call(rows=1 << 28, source=1 << 28, codes_t=0, scales_t=0) == INVALID       # more threads than a launch counts


def test_grouped(L):
    call = caller(L.scaled_gemm_grouped_block128,
                  "M N K groups offsets a_fmt a a_scales b_fmt b b_scales b_block_rows alpha c ldc beta out d ldd stream",
                  dict(M=0, N=8, K=64, groups=2, offsets=P, a_fmt=E4M3, a=P, a_scales=P, b_fmt=E5M2, b=P, b_scales=P,
                       b_block_rows=128, alpha=1.0, c=0, ldc=0, beta=0.0, out=BF16, d=P, ldd=8, stream=None))
    assert call() == OK and call(M=8, N=0) == OK and call(M=8, groups=0) == OK
    assert call(a_fmt=MXFP4) == UNSUPPORTED and call(b_fmt=-1) == UNSUPPORTED and call(out=3) == UNSUPPORTED
    assert call(b_block_rows=32) == UNSUPPORTED
    m = dict(M=8)
    assert call(M=-1) == INVALID and call(N=-1) == INVALID and call(K=-32) == INVALID and call(groups=-1) == INVALID
    assert call(**m, K=48) == INVALID and call(**m, K=1 << 23) == UNSUPPORTED
    assert call(M=(1 << 30) + 1) == UNSUPPORTED and call(**m, groups=1025) == UNSUPPORTED
    assert call(**m, N=(1 << 31) - 256, ldd=1 << 31) == INVALID
    assert call(**m, ldd=7) == INVALID and call(**m, d=0) == INVALID and call(**m, d=P + 1) == INVALID
    assert call(**m, offsets=0) == INVALID and call(**m, offsets=P + 2) == INVALID
    assert call(**m, beta=1.0) == INVALID and call(**m, beta=1.0, c=P, ldc=7) == INVALID
    for k in ("a", "b", "a_scales", "b_scales"):
        assert call(**m, **{k: 0}) == INVALID and call(**m, **{k: P + 2}) == INVALID


def test_wgrad(L):
    call = caller(L.scaled_gemm_grouped_wgrad_block128,
                  "M N columns words groups offsets a_fmt a a_scales b_fmt b b_scales alpha c ldc c_group beta out d ldd "
                  "d_group stream",
                  dict(M=0, N=8, columns=256, words=2, groups=2, offsets=P, a_fmt=E4M3, a=P, a_scales=P, b_fmt=E5M2, b=P,
                       b_scales=P, alpha=1.0, c=0, ldc=0, c_group=0, beta=0.0, out=BF16, d=P, ldd=8, d_group=64,
                       stream=None))
    assert call() == OK and call(M=8, N=0) == OK and call(M=8, groups=0) == OK
    assert call(a_fmt=MXFP4) == UNSUPPORTED and call(b_fmt=-1) == UNSUPPORTED and call(out=3) == UNSUPPORTED
    m = dict(M=8)
    for k in ("M", "N", "columns", "words", "groups"):
        assert call(**{k: -128}) == INVALID
    assert call(**m, columns=200) == INVALID and call(**m, columns=1 << 23) == UNSUPPORTED
    assert call(**m, groups=1025) == UNSUPPORTED and call(**m, words=1 << 31) == INVALID
    assert call(M=(1 << 31) - 256, d_group=1 << 40) == INVALID
    assert call(**m, ldd=7) == INVALID and call(**m, d=0) == INVALID and call(**m, d=P + 1) == INVALID
    assert call(**m, d_group=63) == INVALID
    assert call(**m, offsets=0) == INVALID and call(**m, offsets=P + 2) == INVALID
    assert call(**m, beta=1.0) == INVALID and call(**m, beta=1.0, c=P, ldc=7) == INVALID
    for k in ("a", "b", "a_scales", "b_scales"):
        assert call(**m, **{k: 0}) == INVALID and call(**m, **{k: P + 2}) == INVALID


def test_binding_refuses_tensors_of_the_host():
    import torch
    x, q = torch.zeros((4, 64)), torch.zeros((4, 128), dtype=torch.uint8)
    s, o = torch.zeros((1, 4, 4), dtype=torch.uint8), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: bs.rmsnorm_quantize_block128(x), lambda: bs.rmsnorm_quantize_block128(x, fmt=None),
                 lambda: bs.rmsnorm_backward(x, x, x[:, 0]), lambda: bs.fp8_quantize_grouped_block128(x, o),
                 lambda: bs.scaled_gemm_grouped_block128(q, s, q[None], s[None], o),
                 lambda: bs.scaled_gemm_grouped_block128(q, s, q[None], s[None], o, "mxfp4"),
                 lambda: bs.scaled_gemm_grouped_wgrad_block128(q, s, q, s, o)):
        with pytest.raises(ValueError):
            call()
