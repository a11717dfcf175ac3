"""Plain references of the norm and of the grouped block-of-128 operators: numpy, float64, from the
definitions, one row or group at a time; nothing shared with the HIP library."""
from __future__ import annotations

import numpy as np

from . import block128 as b128


def rmsnorm(h, weight, eps: float):
    """(y, rstd) of a float64 matrix."""
    rstd = 1.0 / np.sqrt((h * h).mean(1) + eps)
    return h * rstd[:, None] * (1.0 if weight is None else weight), rstd


def rmsnorm_backward(dy, h, rstd, weight, dh):
    """(dx, dweight, what their rounding errors are counted in): the gradients with rstd as given, and
    (rstd |g|, rstd |xh| mean|g xh|, sum |dy xh|)."""
    xh = h * rstd[:, None]
    g = dy if weight is None else dy * weight
    dx = rstd[:, None] * (g - xh * (g * xh).mean(1, keepdims=True))
    size = (np.abs(rstd[:, None] * g), np.abs(rstd[:, None] * xh) * np.abs(g * xh).mean(1, keepdims=True),
            np.abs(dy * xh).sum(0))
    return dx if dh is None else dx + dh, (dy * xh).sum(0), size


def spans(offsets):
    """(first row, end) of each group."""
    return [(int(a), int(b)) for a, b in zip(offsets[:-1], offsets[1:])]


def columns(sizes):
    """(first column, first word) of each group in a transpose, and past the last one."""
    c = w = 0
    out = []
    for n in sizes:
        out.append((c, w))
        c += b128.up(n, 128)
        w += b128.up(n, 512) // 512
    return out + [(c, w)]


def quantize_transposed(x: np.ndarray, offsets, fmt: str):
    """Codes [k][columns in use] and scale words [words in use][k][4] of the transpose of sorted rows, group
    by group; a block with a non-finite value holds NaN codes to its end."""
    k = x.shape[1]
    at = columns([b - a for a, b in spans(offsets)])
    codes, scales = np.zeros((k, at[-1][0]), np.uint8), np.full((at[-1][1], k, 4), 127, np.uint8)
    for (a, b), (c, w) in zip(spans(offsets), at):
        if a == b:
            continue
        q, s = b128.quantize(np.ascontiguousarray(x[a:b].T), fmt, 1)
        codes[:, c:c + q.shape[1]] = q
        last = b128.up(b - a, 128)
        if q.shape[1] < last:                      # the quantiser pads to 32, a group to 128
            nan = b128.unwords(s, last // 128)[:, -1] == 255
            codes[:, c + q.shape[1]:c + last][nan] = 0x7F
        scales[w:w + s.shape[0]] = s
    return codes, scales


def gemm_grouped(a, sa, a_fmt, b, sb, b_fmt, b_rows, offsets):
    """(D, S) over all rows: the exact products and sum |a b|; zeros in rows of no group."""
    x = b128.dequantize(a, sa, a_fmt, 1)
    d, s = np.zeros((2, a.shape[0], b.shape[1]))
    for e, (i, j) in enumerate(spans(offsets)):
        if i < j:
            y = b128.dequantize(b[e], sb[e], b_fmt, b_rows)
            d[i:j], s[i:j] = x[i:j] @ y.T, np.abs(x[i:j]) @ np.abs(y).T
    return d, s


def gemm_wgrad(a, sa, a_fmt, b, sb, b_fmt, offsets):
    """(D, S): [groups][M][N]."""
    sizes = [j - i for i, j in spans(offsets)]
    at = columns(sizes)
    d, s = np.zeros((2, len(sizes), a.shape[0], b.shape[0]))
    for e, ((c, w), (c1, w1)) in enumerate(zip(at[:-1], at[1:])):
        if c < c1:
            x = b128.dequantize(a[:, c:c1], sa[w:w1], a_fmt, 1)
            y = b128.dequantize(b[:, c:c1], sb[w:w1], b_fmt, 1)
            d[e], s[e] = x @ y.T, np.abs(x) @ np.abs(y).T
    return d, s
