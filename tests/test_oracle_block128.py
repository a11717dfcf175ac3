"""Pins of the block-of-128 and AdamW references (CPU)."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import block128 as ref

FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_exponent_is_the_smallest_that_fits(fmt):
    g = np.random.default_rng(0)
    a = np.concatenate([np.float32(2.0) ** g.uniform(-140, 127, 500).astype(np.float32),
                        np.float32(ref.TOP[fmt]) * np.float32(2.0) ** np.arange(-100, 90, dtype=np.float32)])
    a = np.concatenate([a, np.nextafter(a, np.float32(np.inf)), np.nextafter(a, np.float32(0))])
    for x, e in zip(a.astype(np.float64), ref.exponent(a, fmt)):
        top = Fraction(ref.TOP[fmt])
        assert top * Fraction(2) ** int(e) >= Fraction(x) or e == 127
        assert e == -127 or top * Fraction(2) ** int(e - 1) < Fraction(x)
    assert ref.exponent(0.0, fmt) == 0 and ref.exponent(ref.TOP[fmt], fmt) == 0


def test_scale_words():
    e = np.arange(2 * 5, dtype=np.uint8).reshape(2, 5)
    w = ref.words(e)
    assert w.shape == (2, 2, 4)
    assert w[0].tolist() == [[0, 1, 2, 3], [5, 6, 7, 8]]
    assert w[1].tolist() == [[4, 127, 127, 127], [9, 127, 127, 127]]
    assert np.array_equal(ref.unwords(w, 5), e)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantizer_matches_torchs_casts(fmt, block_rows):
    g = np.random.default_rng(1)
    x = (g.standard_normal((130, 200)) * 2.0 ** g.integers(-20, 20, (130, 1))).astype(np.float32)
    codes, scales = ref.quantize(x, fmt, block_rows)
    e = ref.unwords(scales, 2).astype(np.int64) - 127
    s = np.repeat(np.repeat(e, block_rows, 0)[:130], 128, 1)[:, :200]
    want = torch.from_numpy(np.ldexp(x, -s).astype(np.float32)).to(FP8[fmt]).view(torch.uint8).numpy()
    assert np.array_equal(codes[:, :200], want) and not codes[:, 200:].any()
    # the transpose of 128 x 128 blocks has the same codes
    if block_rows == 128:
        ct, st = ref.quantize(np.ascontiguousarray(x.T), fmt, 128)
        assert np.array_equal(ct[:, :130].T, codes[:, :200])
        assert np.array_equal(ref.unwords(st, 2).T, ref.unwords(scales, 2))


def test_non_finite_blocks():
    x = np.ones((2, 300), dtype=np.float32)
    x[0, 130], x[1, 299] = np.inf, np.nan
    codes, scales = ref.quantize(x, "e4m3", 1)
    s = ref.unwords(scales, 3)
    assert (s == 255).tolist() == [[False, True, False], [False, False, True]]
    assert np.all(codes[0, 128:256] == 0x7F) and np.isnan(ref.dequantize(codes, scales, "e4m3", 1)[1, 256:]).all()


def test_gemm_against_exact_rationals():
    g = np.random.default_rng(2)
    a, sa = ref.quantize(g.standard_normal((3, 160)).astype(np.float32), "e4m3", 1)
    b, sb = ref.quantize(g.standard_normal((130, 160)).astype(np.float32), "e5m2", 128)
    d, s = ref.gemm(a, sa, "e4m3", 1, b, sb, "e5m2", 128)
    va = torch.from_numpy(a).view(FP8["e4m3"]).double().numpy()
    vb = torch.from_numpy(b).view(FP8["e5m2"]).double().numpy()
    for i, j in ((0, 0), (2, 127), (1, 128), (2, 129)):
        want = sum(Fraction(va[i, k]) * Fraction(2) ** (int(sa[0, i, k // 128]) - 127)
                   * Fraction(vb[j, k]) * Fraction(2) ** (int(sb[0, j // 128, k // 128]) - 127) for k in range(160))
        assert abs(Fraction(d[i, j]) - want) <= Fraction(2) ** -45 * Fraction(s[i, j])


def test_noise_is_even():
    b = ref.noise(1 << 17, 7, 3, 0)
    lo, hi = (b & np.uint64(0xFFFF)).astype(np.float64), (b >> np.uint64(16)).astype(np.float64)
    # 2^17 draws of a uniform on [0, 2^16): the mean's standard deviation is 2^16 / sqrt(12 2^17) = 52
    assert abs(lo.mean() - 32767.5) < 5 * 53 and abs(hi.mean() - 32767.5) < 5 * 53
    assert not np.array_equal(b, ref.noise(1 << 17, 7, 4, 0)) and not np.array_equal(b, ref.noise(1 << 17, 7, 3, 1))


def test_stochastic_rounding_is_unbiased_and_neighbouring():
    g = np.random.default_rng(3)
    x = np.abs(g.standard_normal(128) * 10.0 ** g.uniform(-6, 0, 128)).astype(np.float32)
    total, n = np.zeros(128), 4096
    for i in range(n):
        codes, scales = ref.round_state(x, (g.integers(0, 1 << 16, 128)).astype(np.uint64), False)
        got = ref.state_values(codes, scales)
        total += got
        lo, hi = ref.round_state(x, np.zeros(128, np.uint64), False), ref.round_state(x, np.full(128, 65535, np.uint64), False)
        if i == 0:
            low, high = ref.state_values(*lo), ref.state_values(*hi)
            assert np.all(low <= x) and np.all(x <= high)
        assert np.all((got == low) | (got == high))
    # the mean of n two-point draws lies within 6 standard deviations, at most step / (2 sqrt(n)) each,
    # plus the 2^-16 of a step to which the draws are cut
    assert np.all(np.abs(total / n - x) <= (high - low) * (6 / (2 * np.sqrt(n)) + 2.0 ** -16))


def test_adamw_matches_torchs_optimizer():
    g = np.random.default_rng(4)
    p0, grads = g.standard_normal(50), [g.standard_normal(50) for _ in range(5)]
    t = torch.from_numpy(p0.copy()).requires_grad_()
    opt = torch.optim.AdamW([t], lr=1e-2, betas=(0.9, 0.99), eps=1e-6, weight_decay=0.1, foreach=False)
    p, m, v = p0, np.zeros(50), np.zeros(50)
    hp = dict(lr=1e-2, beta1=0.9, beta2=0.99, eps=1e-6, weight_decay=0.1)
    for i, gr in enumerate(grads):
        t.grad = torch.from_numpy(gr.copy())
        opt.step()
        p, m, v, _ = ref.adamw(p, gr, m, v, hp, i + 1, 1.0, np.float64)
    assert np.allclose(p, t.detach().numpy(), rtol=1e-12, atol=1e-13)


def test_round_bf16():
    x = np.array([1.0, 1.0 + 2.0 ** -8, -1.0 - 2.0 ** -8], dtype=np.float32)
    assert ref.round_bf16(x, np.zeros(3, np.uint64)).tolist() == [1.0, 1.0, -1.0]
    assert ref.round_bf16(x, np.full(3, 0x8000, np.uint64)).tolist() == [1.0, 1.0 + 2.0 ** -7, -1.0 - 2.0 ** -7]


@pytest.mark.parametrize("block_rows", [1, 128])
def test_padding_codes(block_rows):
    """Columns k .. kp - 1: zeros, but NaN codes in a block with a non-finite value."""
    x = np.ones((130, 140), dtype=np.float32)
    x[1, 139] = np.inf
    codes, scales = ref.quantize(x, "e4m3", block_rows)
    bad = np.arange(130) // block_rows == 1 // block_rows
    assert codes.shape == (130, 160) and np.all(codes[bad, 128:] == 0x7F) and not codes[~bad, 140:].any()
