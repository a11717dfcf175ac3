"""The norm's reciprocal root is rounded once (MI355X).

Rows of four integers times a power of two have an exact mean square in FP32, so that rstd is off by its own
rounding alone: half a step, and what is left of the estimate's error (2^-23, relative) after one step of
Newton's method, 3/8 2^-46, with the rounding of the difference, 2^-24 2^-22: below 2^-18 of a step (2^-24) together.
"""
import numpy as np
import pytest

import block_scaled_precision_fp8_amd as bs
from gpu_common import from_dev, say, to_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("power", [0, 1, 7, 40, 55, -20, -49, -50, -51, -66])
def test_rstd_is_the_nearest_value(power):
    g = np.random.default_rng(100 + power)
    x = g.integers(0, 64, (20000, 4)).astype(np.float32)
    x[:, 0] += 1
    say(f"rmsnorm: reciprocal roots, integers times 2^{power}")
    x *= np.float32(2.0 ** power)
    mean = np.square(x.astype(np.float64)).sum(1) / 4
    assert np.array_equal(mean, mean.astype(np.float32))
    got = from_dev(bs.rmsnorm_quantize_block128(to_dev(x), y="f32", rstd=True, eps=0.0).rstd).astype(np.float64)
    want = 1.0 / np.sqrt(mean)
    step = np.spacing(want.astype(np.float32)).astype(np.float64)
    off = float((np.abs(got - want) / step).max())
    say(f"off by up to {off:.4f} of a step")
    assert off <= 0.5 + 2.0 ** -18


def test_zero_infinity_and_nan():
    x = np.array([[0, 0, 0, 0], [np.inf, 1, 1, 1], [np.nan, 1, 1, 1], [3e38, 0, 0, 0], [1, 1, 1, 1]], np.float32)
    say("rmsnorm: reciprocal roots at the ends")
    got = from_dev(bs.rmsnorm_quantize_block128(to_dev(x), y="f32", rstd=True, eps=0.0).rstd)
    assert got[0] == np.inf and got[1] == 0 and np.isnan(got[2]) and got[3] == 0 and got[4] == 1
    got = from_dev(bs.rmsnorm_quantize_block128(to_dev(x), y="f32", rstd=True, eps=4.0).rstd)
    assert got[0] == 0.5 and got[1] == 0 and np.isnan(got[2])
