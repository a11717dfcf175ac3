"""Plain references of the block-of-128 FP8 quantiser and GEMM and of the AdamW step.

Test infrastructure like the rest of this package: numpy, float64 throughout (the AdamW
step also in float32, operation by operation, for bit comparisons), from the definitions;
it shares nothing with the HIP library.
"""
from __future__ import annotations

import numpy as np

from . import decode_table, encode

TOP = {"e4m3": 448.0, "e5m2": 57344.0}


def exponent(amax, fmt: str) -> np.ndarray:
    """Smallest e with TOP 2^e >= amax (0 for 0), clamped to [-127, 127]: by search."""
    amax = np.asarray(amax, dtype=np.float64)
    e = np.full(amax.shape, -127, dtype=np.int64)
    for _ in range(255):
        e = np.where((np.ldexp(TOP[fmt], e) < amax) & (e < 127), e + 1, e)
    return np.where(amax == 0, 0, e)


def up(n: int, m: int) -> int:
    return (n + m - 1) // m * m


def words(e: np.ndarray) -> np.ndarray:
    """Scale bytes [scale rows][K blocks] -> [ceil(K blocks / 4)][scale rows][4], 127 unused."""
    R, nkb = e.shape
    w = np.full((R, up(nkb, 4)), 127, dtype=np.uint8)
    w[:, :nkb] = e
    return np.ascontiguousarray(w.reshape(R, -1, 4).transpose(1, 0, 2))


def unwords(w: np.ndarray, nkb: int) -> np.ndarray:
    return w.transpose(1, 0, 2).reshape(w.shape[1], -1)[:, :nkb]


def quantize(x: np.ndarray, fmt: str, block_rows: int):
    """Codes rows x up(k, 32) and scale words of a float32 matrix."""
    rows, k = x.shape
    x = x.astype(np.float64)
    bad = ~np.isfinite(x)
    edges_r, edges_k = np.arange(0, rows, block_rows), np.arange(0, k, 128)

    def per_block(f, v):
        return f.reduceat(f.reduceat(v, edges_r, 0), edges_k, 1)

    def spread(v):
        return np.repeat(np.repeat(v, block_rows, 0)[:rows], 128, 1)[:, :k]

    e = exponent(per_block(np.maximum, np.abs(np.where(bad, 0.0, x))), fmt)
    nan = per_block(np.logical_or, bad)
    codes = np.zeros((rows, up(k, 32)), dtype=np.uint8)
    codes[:, :k] = encode(fmt, np.ldexp(np.where(bad, 0.0, x), -spread(e))).reshape(rows, k)
    # a block with an infinity or a NaN: NaN scale, NaN codes (its padding columns too)
    wide = np.repeat(np.repeat(nan, block_rows, 0)[:rows], 128, 1)[:, :codes.shape[1]]
    codes[wide] = 0x7F
    return codes, words(np.where(nan, 255, e + 127).astype(np.uint8))


def scale_values(bytes_: np.ndarray) -> np.ndarray:
    b = bytes_.astype(np.int64)
    return np.where(b == 255, np.nan, np.ldexp(1.0, b - 127))


def dequantize(codes: np.ndarray, scales: np.ndarray, fmt: str, block_rows: int) -> np.ndarray:
    rows, K = codes.shape
    s = scale_values(unwords(scales, up(K, 128) // 128))
    s = np.repeat(np.repeat(s, block_rows, 0)[:rows], 128, 1)[:, :K]
    return decode_table(fmt)[codes] * s


def gemm(a, sa, a_fmt, a_rows, b, sb, b_fmt, b_rows):
    """(D, S): the exact product and sum_k |a b|, float64."""
    x, y = dequantize(a, sa, a_fmt, a_rows), dequantize(b, sb, b_fmt, b_rows)
    return x @ y.T, np.abs(x) @ np.abs(y).T


# ---------------------------------------------------------------------------- AdamW
def _mix(h):
    h = np.asarray(h, dtype=np.uint64)
    m = np.uint64(0xFFFFFFFF)
    h = h ^ (h >> np.uint64(16))
    h = (h * np.uint64(0x85EBCA6B)) & m
    h = h ^ (h >> np.uint64(13))
    h = (h * np.uint64(0xC2B2AE35)) & m
    return h ^ (h >> np.uint64(16))


def noise(n: int, seed: int, step: int, index: int) -> np.ndarray:
    """The 32 random bits of each element of tensor `index`."""
    m = np.uint64(0xFFFFFFFF)
    key = _mix(_mix(_mix(seed) ^ np.uint64(step & 0xFFFFFFFF)) ^ np.uint64(index))
    q = np.arange(up(n, 8) // 8, dtype=np.uint64)
    s = _mix((q * np.uint64(0x9E3779B1) + key) & m) | np.uint64(1)
    cols = [s]
    for _ in range(7):
        s = s ^ ((s << np.uint64(13)) & m)
        s = s ^ (s >> np.uint64(17))
        s = s ^ ((s << np.uint64(5)) & m)
        cols.append(s)
    return np.stack(cols, 1).reshape(-1)[:n]


def round_state(x: np.ndarray, bits16: np.ndarray, keep: bool):
    """Stochastic E4M3 codes and scale bytes of a vector; blocks of 128."""
    n = x.size
    codes, scales = np.zeros(n, dtype=np.uint8), np.zeros(up(n, 128) // 128, dtype=np.uint8)
    for j in range(scales.size):
        c = slice(128 * j, min(128 * j + 128, n))
        b = x[c].astype(np.float64)
        if not np.all(np.isfinite(b)):
            scales[j], codes[c] = 255, 0x7F
            continue
        e = int(exponent(np.abs(b).max(), "e4m3"))
        scales[j] = e + 127
        y = np.ldexp(np.abs(b), -e)
        step = np.ldexp(1.0, np.maximum(np.frexp(y)[1] - 1, -6) - 3)
        t = np.floor(np.floor(y / step * 2.0 ** 20) + bits16[c].astype(np.float64) * 16) // 2 ** 20
        if keep:
            t = np.where((b > 0) & (t == 0), 1, t)
        codes[c] = encode("e4m3", np.copysign(t * step, b))
    return codes, scales


def state_values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    return decode_table("e4m3")[codes] * np.repeat(scale_values(scales), 128)[:codes.size]


def round_bf16(x: np.ndarray, bits16: np.ndarray) -> np.ndarray:
    """float32 -> bf16 (as float32), the 16 cut bits carrying with bits16."""
    w = x.astype(np.float32).view(np.uint32).astype(np.uint64)
    return ((w + bits16) & np.uint64(0xFFFF0000)).astype(np.uint32).view(np.float32)


def constants(lr, beta1, beta2, eps, weight_decay, step):
    return (beta1, 1 - beta1, beta2, 1 - beta2, 1 - lr * weight_decay, lr / (1 - beta1 ** step),
            1 / np.sqrt(1 - beta2 ** step), eps)


def adamw(p, g, m, v, hp, step, grad_scale, dtype):
    """(p', m', v', sqrt(v')) of one step; every operation rounded to `dtype`."""
    b1, c1, b2, c2, decay, size, rbc, eps = (dtype(c) for c in constants(**hp, step=step))
    p, g, m, v = (np.asarray(t).astype(dtype) for t in (p, g, m, v))
    g = g * dtype(grad_scale)
    m = b1 * m + c1 * g
    v = b2 * v + (c2 * g) * g
    r = np.sqrt(v)
    return p * decay - (size * m) / (r * rbc + eps), m, v, r
