"""Pins of the float64 references of the norm and of the grouped operators (CPU): against torch's
autograd, central differences, and products written out row by row."""
import numpy as np
import pytest

from oracle import block128 as b128
from oracle import experts as ref


@pytest.mark.parametrize("rows,k,weighted,residual", [(1, 1, True, False), (3, 7, False, True), (5, 130, True, True)])
def test_norm_gradients(rows, k, weighted, residual):
    import torch
    g = np.random.default_rng(rows * 100 + k)
    h, dy, dh = g.standard_normal((3, rows, k))
    w = g.standard_normal(k) if weighted else None
    eps = 1e-3
    th = torch.tensor(h, requires_grad=True)
    tw = torch.tensor(w if weighted else np.ones(k), requires_grad=True)
    ty = th * torch.rsqrt(th.square().mean(1, keepdim=True) + eps) * tw
    loss = (ty * torch.tensor(dy)).sum() + ((th * torch.tensor(dh)).sum() if residual else 0)
    loss.backward()
    y, rstd = ref.rmsnorm(h, w, eps)
    np.testing.assert_allclose(y, ty.detach().numpy(), rtol=1e-12)
    dx, dw, _ = ref.rmsnorm_backward(dy, h, rstd, w, dh if residual else None)
    np.testing.assert_allclose(dx, th.grad.numpy(), rtol=1e-9, atol=1e-12)
    np.testing.assert_allclose(dw, tw.grad.numpy(), rtol=1e-9, atol=1e-12)
    # central differences: error O(step^2) of the third derivative and 2^-52 / step of the values
    step = 1e-4
    for i, j in [(0, 0), (rows - 1, k // 2)]:
        up, down = h.copy(), h.copy()
        up[i, j] += step
        down[i, j] -= step
        f = [(ref.rmsnorm(v, w, eps)[0] * dy).sum() + ((v * dh).sum() if residual else 0) for v in (up, down)]
        assert abs((f[0] - f[1]) / (2 * step) - dx[i, j]) < 1e-4 * (1 + abs(dx[i, j]))


def test_columns_and_words():
    assert ref.columns([0, 1, 128, 129, 513]) == [(0, 0), (0, 0), (128, 1), (256, 2), (512, 3), (1152, 5)]


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_transposed_groups_hold_each_groups_transpose(fmt):
    g = np.random.default_rng(3)
    offsets = [0, 0, 5, 133, 133, 700]
    x = (g.standard_normal((700, 9)) * np.exp2(g.integers(-6, 6, (700, 1)))).astype(np.float32)
    codes, scales = ref.quantize_transposed(x, offsets, fmt)
    at = ref.columns([b - a for a, b in ref.spans(offsets)])
    assert codes.shape == (9, at[-1][0]) and scales.shape == (at[-1][1], 9, 4)
    step = 2.0 ** -4 if fmt == "e4m3" else 2.0 ** -3            # half a step, relative
    for (a, b), (c, w), (_, w1) in zip(ref.spans(offsets), at, at[1:]):
        if a == b:
            continue
        v = b128.dequantize(codes[:, c:c + b128.up(b - a, 128)], scales[w:w1], fmt, 1)
        assert not v[:, b - a:].any()
        amax = np.abs(v).max()
        assert (np.abs(v[:, :b - a] - x[a:b].T) <= step * np.abs(x[a:b].T) + 2.0 ** -8 * amax).all()


def test_products():
    g = np.random.default_rng(4)
    offsets = [1, 3, 3, 8]
    x, w = g.standard_normal((9, 64)).astype(np.float32), g.standard_normal((3, 5, 64)).astype(np.float32)
    a, sa = b128.quantize(x, "e4m3", 1)
    b, sb = zip(*[b128.quantize(v, "e5m2", 128) for v in w])
    d, s = ref.gemm_grouped(a, sa, "e4m3", np.stack(b), np.stack(sb), "e5m2", 128, offsets)
    va = b128.dequantize(a, sa, "e4m3", 1)
    for i in range(9):
        e = {1: 0, 2: 0}.get(i, 2 if 3 <= i < 8 else None)
        for n in range(5):
            want = 0.0 if e is None else float(np.dot(va[i], b128.dequantize(b[e], sb[e], "e5m2", 128)[n]))
            assert abs(d[i, n] - want) <= 1e-12 * (1 + s[i, n])
    y = g.standard_normal((9, 4)).astype(np.float32)
    (qx, sx), (qy, sy) = ref.quantize_transposed(x[1:8], [0, 2, 2, 7], "e4m3"), ref.quantize_transposed(y[1:8], [0, 2, 2, 7], "e5m2")
    d, s = ref.gemm_wgrad(qy, sy, "e5m2", qx, sx, "e4m3", [0, 2, 2, 7])
    assert d.shape == (3, 4, 64) and not d[1].any()
    # each code is within half a step of its element, relative (2^-4, 2^-3) or to its block's largest
    for e, (i, j) in enumerate([(1, 3), (3, 3), (3, 8)]):
        exact = y[i:j].T.astype(np.float64) @ x[i:j]
        assert (np.abs(d[e] - exact) <= (2.0 ** -3 + 2.0 ** -4 + 2.0 ** -6) * (np.abs(y[i:j]).T @ np.abs(x[i:j])) + 1e-2).all()
