"""The grouped block-of-128 operators against their float64 references (MI355X).

Quantiser: byte-equal.  Products: |D - D_ref| <= tol(K) (|alpha| S + |beta C|), S = sum |a b|, with the
tolerance of the ungrouped product: 16-bit outputs lose up to 7 2^-13 of S in the FP8 instruction and one
rounding per 16 products twice, FP32 output 8 2^-24 and one rounding per 8 products twice; up to 16
partial sums of split K, alpha, beta and the output's half step come on top.  From 65520 on, half a
step above its largest value 65504, FP16 rounds to infinity, so a value within its bound of that or
beyond it may be infinite.
"""
import numpy as np
import pytest

import block_scaled_precision_fp8_amd as bs
from gpu_common import from_dev, guarded, say, untouched
from oracle import block128 as b128
from oracle import experts as ref

pytestmark = pytest.mark.gpu

HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 0.0, "bf16": 0.0, "f16": 2.0 ** -25}


def tol(out, K):
    if out == "f32":
        return (8 + 2 * K / 8 + 16 + 2) * 2.0 ** -24 + HALF[out]
    return 7 * 2.0 ** -13 + (2 * K / 16 + 16 + 2) * 2.0 ** -24 + HALF[out]


def dtype(t):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[t]


def values(rows, k, seed, spread=4):
    g = np.random.default_rng(seed)
    x = g.standard_normal((rows, k)) * np.exp2(g.integers(-spread, spread + 1, (rows, 1)))
    x *= np.exp2(g.integers(-2, 3, (1, k)))
    x[g.random((rows, k)) < 0.05] = 0
    return x.astype(np.float32)


def dev(a, t=None):
    import torch
    x = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return x if t is None else x.to(dtype(t))


def offs(sizes, first=0):
    import torch
    o = np.concatenate([[first], first + np.cumsum(sizes)]).astype(np.int32)
    return o, torch.from_numpy(o).cuda()


#: sizes of groups: empty ones first, last and in a row; around the tile sizes; more than 64 groups
GROUPS = [[1], [0, 1, 0], [128, 1, 127], [129, 0, 0, 513, 16, 17], [0, 300, 5, 64, 65], [3] * 7 + [0] * 70 + [2, 40],
          [700, 31, 33, 32]]


# ------------------------------------------------------------------ quantiser
@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("g,sizes", enumerate(GROUPS))
def test_quantize(g, sizes, t):
    import torch
    k = (1, 40, 128, 257, 600, 33, 1000)[g]
    o, od = offs(sizes)
    n = int(o[-1])
    src = dev(values(n, k, g), t)
    r = np.random.default_rng(g)
    fmt = ("e4m3", "e5m2")[g % 2]
    for index in (None, r.integers(0, n, n).astype(np.int32)):
        x = from_dev(src) if index is None else from_dev(src)[index]
        di = None if index is None else dev(index)
        for want in ("both", "rows", "transposed"):
            say(f"quantize_grouped {sizes[:6]} k {k} {t} {fmt} {want} index {index is not None}")
            got = bs.fp8_quantize_grouped_block128(src, od, fmt, di, rows=want != "transposed", transposed=want != "rows")
            if want != "transposed":
                codes, scales = b128.quantize(x, fmt, 1)
                assert np.array_equal(from_dev(got[0]), codes) and np.array_equal(from_dev(got[1]), scales)
            if want != "rows":
                codes, scales = ref.quantize_transposed(x, o, fmt)
                assert np.array_equal(from_dev(got[-2])[:, :codes.shape[1]], codes)
                assert np.array_equal(from_dev(got[-1])[:scales.shape[0]], scales)


def test_quantize_index_outside_and_rows_of_no_group():
    """Indexes outside x stand for zeros; rows before the first and after the last group, and columns past
    the last one, are left as they were."""
    import torch
    say("quantize_grouped: indexes outside, rows of no group")
    x = values(20, 300, 1)
    index = np.array([3, -1, 19, 20, 0, 1 << 30, -(1 << 31), 7] * 5, np.int32)
    o, od = offs([7, 0, 21], first=4)
    xs = np.where(((index >= 0) & (index < 20))[:, None], x[np.clip(index, 0, 19)], 0).astype(np.float32)
    (k, cols), (words, _, _) = bs.block128_grouped_shape(40, 300, 3)
    shapes = [(40, 320), (1, 40, 4), (k, cols), (words, k, 4)]
    bufs = [guarded((int(np.prod(s)),), torch.uint8, tail=64) for s in shapes]
    outs = [v.view(s) for (_, v), s in zip(bufs, shapes)]
    for want in (True, False):
        if want:
            bs.fp8_quantize_grouped_block128(dev(x), od, "e4m3", dev(index), True, True, *outs)
        else:
            outs[0].fill_(0xA5), outs[1].fill_(0xA5)
            bs.fp8_quantize_grouped_block128(dev(x), od, "e4m3", dev(index), True, False, *outs[:2])
        codes, scales = b128.quantize(xs, "e4m3", 1)
        got, gs = from_dev(outs[0]), from_dev(outs[1])
        assert np.array_equal(got[4:32], codes[4:32]) and np.array_equal(gs[:, 4:32], scales[:, 4:32])
        for a in (got[:4], got[32:], gs[:, :4], gs[:, 32:]):
            assert (a == 0xA5).all()
    codes, scales = ref.quantize_transposed(xs[4:32], o - 4, "e4m3")
    got, gs = from_dev(outs[2]), from_dev(outs[3])
    assert np.array_equal(got[:, :codes.shape[1]], codes) and (got[:, codes.shape[1]:] == 0xA5).all()
    assert np.array_equal(gs[:2], scales) and (gs[2:] == 0xA5).all()
    assert all(untouched(b, (int(np.prod(s)),), tail=64) for (b, _), s in zip(bufs, shapes))


def test_quantize_non_finite_blocks():
    import torch
    say("quantize_grouped: non-finite blocks")
    x = values(300, 70, 2)
    x[5, 3], x[200, 60], x[299, 69] = np.nan, np.inf, -np.inf
    o, od = offs([10, 150, 140])
    got = [from_dev(t) for t in bs.fp8_quantize_grouped_block128(dev(x), od, "e5m2", transposed=True)]
    want = [*b128.quantize(x, "e5m2", 1), *ref.quantize_transposed(x, o, "e5m2")]
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    assert np.array_equal(got[2][:, :want[2].shape[1]], want[2]) and np.array_equal(got[3][:want[3].shape[0]], want[3])


@pytest.mark.parametrize("off,extra", [(0, 8), (1, 0), (0, 3)])
@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_quantize_strides(t, off, extra):
    import torch
    n, k = 140, 200
    v = dev(values(n, k, 3), t)
    base = torch.zeros(n * (k + extra) + off + 8, dtype=v.dtype, device="cuda")
    view = base[off:off + n * (k + extra)].view(n, k + extra)[:, :k]
    view.copy_(v)
    _, od = offs([100, 40])
    say(f"quantize_grouped view offset {off} extra {extra} {t}")
    for rows, transposed in ((True, False), (True, True)):
        a = bs.fp8_quantize_grouped_block128(view, od, transposed=transposed)
        b = bs.fp8_quantize_grouped_block128(v, od, transposed=transposed)
        cols = 256
        assert a[0].equal(b[0]) and a[1].equal(b[1])
        if transposed:
            assert a[2][:, :cols].equal(b[2][:, :cols]) and a[3][:2].equal(b[3][:2])


# ------------------------------------------------------------------ products of rows
def weights(E, N, K, fmt, rows, seed):
    w = [b128.quantize(values(N, K, seed + e, 2), fmt, rows) for e in range(E)]
    return np.stack([c for c, _ in w]), np.stack([s for _, s in w])


def check(d, want, s, out, K, label, alpha=1.0, beta=0.0, c=None):
    d = from_dev(d).astype(np.float64)
    r, m = alpha * want, abs(alpha) * s
    if c is not None:
        r, m = r + beta * c, m + np.abs(beta * c)
    lim = tol(out, K) * m + TINY[out]
    over = (out == "f16") & np.isinf(d) & (np.abs(r) + lim >= 65520) & (np.sign(d) == np.sign(r))
    err = np.abs(np.where(over, r, d) - r)
    worst = float((err / np.maximum(lim, 1e-300)).max()) if d.size else 0.0
    say(f"{label}: {worst:.3f} of the bound")
    assert (err <= lim).all(), f"{label}: {worst:.3f} of the bound"


SIZES = [(1, 32), (16, 128), (40, 160), (130, 512), (256, 544), (70, 1056), (129, 2048)]


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("g,sizes", enumerate(GROUPS))
def test_grouped(g, sizes, out):
    import torch
    N, K = SIZES[g]
    af, bf, br = ("e4m3", "e5m2")[g % 2], ("e4m3", "e5m2")[(g // 2) % 2], (1, 128)[(g + 1) % 2]
    o, od = offs(sizes, first=3)
    M = int(o[-1]) + 5
    a, sa = b128.quantize(values(M, K, 10 + g), af, 1)
    b, sb = weights(len(sizes), N, K, bf, br, 100 * g)
    want, s = ref.gemm_grouped(a, sa, af, b, sb, bf, br, o)
    args = [dev(v) for v in (a, sa, b, sb)] + [od, af, bf, br]
    inside = np.zeros(M, bool)
    inside[3:o[-1]] = True
    for alpha, beta, extra in ((1.0, 0.0, 0), (0.5, 0.0, 3), (1.0, 1.0, 0), (-2.0, 0.5, 8)):
        label = f"grouped {sizes[:6]} N {N} K {K} {af} {bf} block rows {br} {out} alpha {alpha} beta {beta} extra {extra}"
        say(label)
        buf, d = guarded((M, N), dtype(out), extra_cols=extra, extra_rows=1, tail=16)
        before = d.clone()
        c = None if beta == 0.0 else dev(values(M, N, 77, 0), out)
        bs.scaled_gemm_grouped_block128(*args, out=out, alpha=alpha, c=c, beta=beta, d=d)
        ii = torch.from_numpy(inside).cuda()
        check(d[ii], want[inside], s[inside], out, K, label, alpha, beta,
              None if c is None else from_dev(c).astype(np.float64)[inside])
        bits = {4: torch.int32, 2: torch.int16}[d.element_size()]
        assert d[~ii].view(bits).equal(before[~ii].view(bits))
        assert untouched(buf, (M, N), extra, 1, 16)
        if beta == 1.0:
            d2 = c.clone()                         # in place
            bs.scaled_gemm_grouped_block128(*args, out=out, alpha=alpha, c=d2, beta=beta, d=d2)
            assert d2[ii].equal(d[ii])


def test_grouped_without_k():
    import torch
    say("grouped, K = 0")
    _, od = offs([2, 0, 1], first=1)
    u8 = dict(dtype=torch.uint8, device="cuda")
    a, sa, b, sb = torch.zeros((5, 0), **u8), torch.zeros((0, 5, 4), **u8), torch.zeros((3, 9, 0), **u8), torch.zeros((3, 0, 1, 4), **u8)
    d = torch.full((5, 9), 3.0, device="cuda")
    bs.scaled_gemm_grouped_block128(a, sa, b, sb, od, out="f32", alpha=2.0, c=d, beta=0.5, d=d)
    assert d.cpu().tolist() == [[3.0] * 9] + [[1.5] * 9] * 3 + [[3.0] * 9]
    bs.scaled_gemm_grouped_block128(a, sa, b, sb, od, out="f32", d=d)
    assert d.cpu().tolist() == [[3.0] * 9] + [[0.0] * 9] * 3 + [[3.0] * 9]


# ------------------------------------------------------------------ products over rows
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("g,sizes", enumerate(GROUPS))
def test_wgrad(g, sizes, out):
    import torch
    M, N = ((1, 1), (40, 33), (130, 64), (64, 260), (200, 31), (16, 48), (257, 129))[g]
    af, bf = ("e4m3", "e5m2")[(g + 1) % 2], ("e4m3", "e5m2")[(g // 2) % 2]
    o, od = offs(sizes)
    n = int(o[-1])
    qa, sa = bs.fp8_quantize_grouped_block128(dev(values(n, M, 20 + g, 2)), od, af, rows=False, transposed=True)
    qb, sb = bs.fp8_quantize_grouped_block128(dev(values(n, N, 30 + g, 2)), od, bf, rows=False, transposed=True)
    want, s = ref.gemm_wgrad(from_dev(qa), from_dev(sa), af, from_dev(qb), from_dev(sb), bf, o)
    E = len(sizes)
    for alpha, beta, extra in ((1.0, 0.0, 0), (0.5, 0.0, 3), (1.0, 1.0, 0), (-2.0, 0.5, 8)):
        label = f"wgrad {sizes[:6]} M {M} N {N} {af} {bf} {out} alpha {alpha} beta {beta} extra {extra}"
        say(label)
        buf, flat = guarded((E * (M + 1), N), dtype(out), extra_cols=extra, extra_rows=1, tail=16)
        d = flat.unflatten(0, (E, M + 1))[:, :M]
        edge = flat.unflatten(0, (E, M + 1))[:, M].clone()
        c = None if beta == 0.0 else dev(values(E * M, N, 78, 0), out).view(E, M, N)
        bs.scaled_gemm_grouped_wgrad_block128(qa, sa, qb, sb, od, af, bf, out=out, alpha=alpha, c=c, beta=beta, d=d)
        check(d, want, s, out, max(sizes) + 128, label, alpha, beta, None if c is None else from_dev(c).astype(np.float64))
        bits = {4: torch.int32, 2: torch.int16}[d.element_size()]
        assert flat.unflatten(0, (E, M + 1))[:, M].view(bits).equal(edge.view(bits))
        assert untouched(buf, (E * (M + 1), N), extra, 1, 16)
        if beta == 1.0:
            d2 = c.clone()
            bs.scaled_gemm_grouped_wgrad_block128(qa, sa, qb, sb, od, af, bf, out=out, alpha=alpha, c=d2, beta=beta, d=d2)
            assert d2.equal(d)


def test_wgrad_without_rows():
    import torch
    say("wgrad without rows")
    od = torch.zeros(4, dtype=torch.int32, device="cuda")
    u8 = dict(dtype=torch.uint8, device="cuda")
    a, sa, b, sb = torch.zeros((5, 0), **u8), torch.zeros((0, 5, 4), **u8), torch.zeros((6, 0), **u8), torch.zeros((0, 6, 4), **u8)
    d = torch.full((3, 5, 6), 3.0, device="cuda")
    bs.scaled_gemm_grouped_wgrad_block128(a, sa, b, sb, od, out="f32", c=d, beta=0.5, d=d)
    assert bool((d == 1.5).all())
    bs.scaled_gemm_grouped_wgrad_block128(a, sa, b, sb, od, out="f32", d=d)
    assert not d.any()


# ------------------------------------------------------------------ offsets that break the rules
@pytest.mark.parametrize("o", [[0, 50, 20, 90], [-7, 30, 60, 90], [0, 200, 300, 400], [90, 60, 30, 0], [5, 5, 5, 5],
                               [0, 2 ** 31 - 1, -(2 ** 31), 90], [-5, -4, -3, -2], [95, 96, 97, 98]])
def test_offsets_that_break_the_rules_stay_inside(o):
    """Whatever the device holds, nothing outside the outputs is written (what is inside is undefined)."""
    import torch
    say(f"offsets {o}")
    od = torch.tensor(o, dtype=torch.int32, device="cuda")
    x = dev(values(90, 300, 1))
    (k, cols), (words, _, _) = bs.block128_grouped_shape(90, 300, 3)
    shapes = [(90, 320), (1, 90, 4), (k, cols), (words, k, 4)]
    bufs = [guarded((int(np.prod(s)),), torch.uint8, tail=4096) for s in shapes]
    outs = [v.view(s) for (_, v), s in zip(bufs, shapes)]
    bs.fp8_quantize_grouped_block128(x, od, "e4m3", None, True, True, *outs)
    bs.fp8_quantize_grouped_block128(x, od, "e4m3", None, True, False, *outs[:2])
    assert all(untouched(b, (int(np.prod(s)),), tail=4096) for (b, _), s in zip(bufs, shapes))
    b, sb = weights(3, 70, 320, "e4m3", 128, 5)
    buf, d = guarded((90, 70), torch.bfloat16, extra_rows=64, tail=64)
    bs.scaled_gemm_grouped_block128(outs[0], outs[1], dev(b), dev(sb), od, d=d)
    assert untouched(buf, (90, 70), 0, 64, 64)
    buf, d = guarded((3 * 300, 300), torch.float32, extra_rows=8)
    bs.scaled_gemm_grouped_wgrad_block128(outs[2], outs[3], outs[2], outs[3], od, out="f32", d=d.view(3, 300, 300))
    assert untouched(buf, (900, 300), 0, 8)


def test_refusals_launch_nothing():
    import torch
    u8 = dict(dtype=torch.uint8, device="cuda")
    o, od = offs([3, 2])
    x = dev(values(5, 64, 1))
    a, sa = bs.fp8_quantize_block128(x)
    b, sb = torch.zeros((2, 8, 64), **u8), torch.zeros((2, 1, 1, 4), **u8)
    qt, st = bs.fp8_quantize_grouped_block128(x, od, rows=False, transposed=True)
    d = torch.full((5, 8), 7.0, dtype=torch.bfloat16, device="cuda")
    g = torch.full((2, 64, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    G, W, Q = bs.scaled_gemm_grouped_block128, bs.scaled_gemm_grouped_wgrad_block128, bs.fp8_quantize_grouped_block128
    bad = [lambda: G(a, sa, b, sb, od.long(), d=d), lambda: G(a, sa, b, sb, od.cpu(), d=d),
           lambda: G(a, sa, b, sb, od[:2], d=d), lambda: G(a, sa, b, sb, od[:0], d=d), lambda: G(a, sa, b, sb, od[None], d=d),
           lambda: G(a, sa[:, :4], b, sb, od, d=d), lambda: G(a, sa, b[:1], sb, od, d=d),
           lambda: G(a, sa, b, sb[:1], od, d=d), lambda: G(a, sa, b, sb, od, b_block_rows=1, d=d),
           lambda: G(a, sa, b[:, :, :32], sb, od, d=d), lambda: G(a, sa, b, sb, od, d=d[:4]),
           lambda: G(a, sa, b, sb, od, out="f32", d=d), lambda: G(a, sa, b, sb, od, beta=1.0, d=d),
           lambda: G(a.view(torch.int8), sa, b, sb, od, d=d), lambda: G(a, sa, b, sb, od, b_block_rows=64, d=d),
           lambda: W(qt, st, qt, st, od.long(), d=g), lambda: W(qt, st, qt[:, :128], st, od, d=g),
           lambda: W(qt, st[:1], qt, st, od, d=g), lambda: W(qt, st, qt[:32], st, od, d=g),
           lambda: W(qt, st, qt, st, od, d=g[:1]), lambda: W(qt, st, qt, st, od, d=g.transpose(1, 2)),
           lambda: W(qt, st, qt, st, od, beta=1.0, d=g), lambda: W(qt, st, qt, st, od, "e3m4", d=g),
           lambda: W(qt, st, qt, st, od, d=g[:1].expand(2, 64, 64)),
           lambda: W(qt[:, :100].contiguous(), st, qt[:, :100].contiguous(), st, od, d=g),
           lambda: Q(x, od.long()), lambda: Q(x, od, index=od.long()), lambda: Q(x, od, index=od.cpu()),
           lambda: Q(x, od, rows=False), lambda: Q(x.double(), od), lambda: Q(x.t(), od), lambda: Q(x, od, "e3m4"),
           lambda: Q(x, od, codes_t=qt), lambda: Q(x, od, transposed=True, codes_t=qt[:, :128]),
           lambda: Q(x, od, transposed=True, scales_t=st[:1]), lambda: Q(x, od, codes=a[:4])]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            print(i)
    assert bool((d == 7.0).all()) and bool((g == 7.0).all())


# ------------------------------------------------------------------ together
def chain(x, residual, w, up, down, index, offsets, dz):
    """One feed-forward step of experts and its gradients: norm, dispatch, two products, and back."""
    f = bs.rmsnorm_quantize_block128(x, w, residual, y="bf16", fmt=None, rstd=True)
    q, s, qt, st = bs.fp8_quantize_grouped_block128(f.y, offsets, "e4m3", index, transposed=True)
    u = bs.scaled_gemm_grouped_block128(q, s, up["q"], up["s"], offsets)
    p, ps, pt, pst = bs.fp8_quantize_grouped_block128(u, offsets, "e4m3", transposed=True)
    z = bs.scaled_gemm_grouped_block128(p, ps, down["q"], down["s"], offsets)
    g, gs, gt, gst = bs.fp8_quantize_grouped_block128(dz, offsets, "e5m2", transposed=True)
    d_down = bs.scaled_gemm_grouped_wgrad_block128(gt, gst, pt, pst, offsets, "e5m2", "e4m3", out="f32")
    du = bs.scaled_gemm_grouped_block128(g, gs, down["qt"], down["st"], offsets, "e5m2")
    h, hs, ht, hst = bs.fp8_quantize_grouped_block128(du, offsets, "e5m2", transposed=True)
    d_up = bs.scaled_gemm_grouped_wgrad_block128(ht, hst, qt, st, offsets, "e5m2", "e4m3", out="f32")
    dy = bs.scaled_gemm_grouped_block128(h, hs, up["qt"], up["st"], offsets, "e5m2", out="f32")
    per_token = dy.new_zeros(f.y.shape).index_add_(0, index.long(), dy)
    dx, dw = bs.rmsnorm_backward(per_token, f.h, f.rstd, w)
    return {"y": f.y, "u": u, "z": z, "d_down": d_down, "d_up": d_up, "du": du, "dx": dx, "dw": dw}


def experts(E, N, K, seed):
    import torch
    w = [dev(values(N, K, seed + e, 0) * 0.05) for e in range(E)]
    parts = [bs.fp8_quantize_block128(v, "e4m3", 128, True, True) for v in w]
    return {k: torch.stack([p[i] for p in parts]) for i, k in enumerate(("q", "s", "qt", "st"))} | {"w": torch.stack(w)}


def test_a_step_of_experts():
    """The operators together against a float64 step with the same dequantised operands at each
    stage's entry: gradients within the FP8 formats' half steps of the exact ones, in the 2-norm."""
    import torch
    tokens, hidden, inner, E = 150, 384, 640, 6
    say("a step of experts")
    x, r = dev(values(tokens, hidden, 1, 0), "bf16"), dev(values(tokens, hidden, 2, 0), "bf16")
    w = dev(1 + 0.1 * values(1, hidden, 3, 0)[0])
    up, down = experts(E, inner, hidden, 10), experts(E, hidden, inner, 20)
    rng = np.random.default_rng(5)
    who = np.stack([rng.permutation(E - 1)[:2] for _ in range(tokens)]).reshape(-1)      # the last expert gets none
    order = np.argsort(who, kind="stable")
    o, od = offs(np.bincount(who, minlength=E))
    index = dev((order // 2).astype(np.int32))
    dz = dev(values(2 * tokens, hidden, 6, 0) * 1e-3, "bf16")
    got = chain(x, r, w, up, down, index, od, dz)
    # the same step without FP8, in float64
    h = (x.float() + r.float()).bfloat16().double()
    rstd = torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-6)
    y = (h * rstd * w.double())[index.long()]
    sp = [slice(a, b) for a, b in ref.spans(o)]
    f = lambda v, m: torch.cat([v[s] @ m[e].double().t() for e, s in enumerate(sp)])     # noqa: E731
    b = lambda v, m: torch.cat([v[s] @ m[e].double() for e, s in enumerate(sp)])         # noqa: E731
    u = f(y, up["w"])
    du = b(dz.double(), down["w"])
    dy = torch.zeros((tokens, hidden), dtype=torch.float64, device="cuda").index_add_(0, index.long(), b(du, up["w"]))
    xh = h * rstd
    gw = dy * w.double()
    want = {"y": h * rstd * w.double(), "u": u, "z": f(u, down["w"]), "du": du,
            "d_down": torch.stack([dz.double()[s].t() @ u[s] for s in sp]),
            "d_up": torch.stack([du[s].t() @ y[s] for s in sp]), "dw": (dy * xh).sum(0),
            "dx": rstd * (gw - xh * (gw * xh).mean(1, keepdim=True))}
    # each quantised operand is within 2^-4 (e4m3) or 2^-3 (e5m2) of its values, relative, or, below its
    # block's smallest normal code, far below the block's largest; in products the errors of elements add up as independent ones do,
    # so that the 2-norm of a result is off by no more than the sum of its operands' bounds
    bound = {"y": 2.0 ** -8, "u": 2 * 2.0 ** -4, "z": 4 * 2.0 ** -4, "du": 2.0 ** -3 + 2.0 ** -4,
             "d_down": 2.0 ** -3 + 3 * 2.0 ** -4, "d_up": 2 * 2.0 ** -3 + 2 * 2.0 ** -4, "dx": 2 * 2.0 ** -3 + 2 * 2.0 ** -4,
             "dw": 2 * 2.0 ** -3 + 2 * 2.0 ** -4}
    for k, v in want.items():
        off = float((got[k].double() - v).norm() / v.norm())
        say(f"{k}: off by {off:.2e}, bound {bound[k]:.2e}")
        assert off <= bound[k], k
    assert not got["d_up"][E - 1].any() and not got["d_down"][E - 1].any()


def test_a_captured_step_follows_new_offsets():
    """A step captured once and replayed with other tokens, indexes and group sizes, on a side stream's warm-up."""
    import torch
    tokens, hidden, inner, E = 60, 256, 320, 5
    up, down = experts(E, inner, hidden, 30), experts(E, hidden, inner, 40)
    w = dev(1 + 0.1 * values(1, hidden, 3, 0)[0])

    def inputs(seed):
        rng = np.random.default_rng(seed)
        who = rng.integers(0, 1 + seed % E, 2 * tokens)
        return (dev(values(tokens, hidden, seed, 0), "bf16"), dev(values(tokens, hidden, seed + 1, 0), "bf16"),
                dev((np.argsort(who, kind="stable") // 2).astype(np.int32)), offs(np.bincount(who, minlength=E))[1],
                dev(values(2 * tokens, hidden, seed + 2, 0), "bf16"))

    say("a captured step of experts")
    x, r, index, od, dz = inputs(4)
    run = lambda: chain(x, r, w, up, down, index, od, dz)        # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for seed in (4, 7, 13, 6):
        for to, v in zip((x, r, index, od, dz), inputs(seed)):
            to.copy_(v)
        graph.replay()
        want = run()
        for k in ("y", "u", "z", "du", "d_down", "d_up"):
            assert out[k].equal(want[k]), (seed, k)


def test_two_streams_at_once():
    import torch
    say("grouped products on two streams")
    E, N, K = 4, 500, 640
    b, sb = (dev(v) for v in weights(E, N, K, "e4m3", 128, 50))
    cases = []
    for i, sizes in enumerate(([3, 0, 5, 1], [200, 100, 0, 300], [40, 41, 42, 43])):
        o, od = offs(sizes)
        x = dev(values(int(o[-1]), K, i), "bf16")
        cases.append((x, od))

    def step(x, od):
        q, s, qt, st = bs.fp8_quantize_grouped_block128(x, od, transposed=True)
        return [bs.scaled_gemm_grouped_block128(q, s, b, sb, od),
                bs.scaled_gemm_grouped_wgrad_block128(qt, st, qt, st, od, out="f32")]

    want = [step(*c) for c in cases]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for i in range(12):
        with torch.cuda.stream(streams[i % 2]):
            got.append(step(*cases[i % 3]))
    torch.cuda.synchronize()
    assert all(a.equal(c) for i, g in enumerate(got) for a, c in zip(g, want[i % 3]))


# ------------------------------------------------------------------ arrays past 2^32 bytes
def test_rows_past_32_bits():
    """Codes and outputs of more than 2^32 bytes: the last group's rows against their own small product."""
    import torch
    M, N, K, E = 280000, 8192, 64, 3
    say("grouped: D past 2^32 bytes")
    o, od = offs([279000, 0, 995], first=2)
    a = torch.randint(0, 0x7E, (M, K), dtype=torch.uint8, device="cuda")
    sa = torch.randint(120, 130, (1, M, 4), dtype=torch.uint8, device="cuda")
    b, sb = (dev(v) for v in weights(E, N, K, "e4m3", 128, 60))
    d = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    bs.scaled_gemm_grouped_block128(a, sa, b, sb, od, d=d)
    for e, (p, q) in ((0, (278500, 279002)), (2, (279002, 279997))):
        want, s = ref.gemm_grouped(from_dev(a[p:q]), from_dev(sa[:, p:q].contiguous()), "e4m3", from_dev(b[e:e + 1]),
                                   from_dev(sb[e:e + 1]), "e4m3", 128, [0, q - p])
        check(d[p:q], want, s, "bf16", K, f"rows {p} .. {q - 1}")
    assert bool((d[:2] == 7.0).all()) and bool((d[279997:] == 7.0).all())


def test_weights_past_32_bits():
    """Experts whose weights lie past 2^32 bytes, in the form for few rows and in a tiled one."""
    import torch
    N, K, E = 32768, 49152, 3
    say("grouped: B past 2^32 bytes")
    b = torch.randint(0, 0x7E, (E, N, K), dtype=torch.uint8, device="cuda")
    sb = torch.randint(120, 130, (E, K // 512, N // 128, 4), dtype=torch.uint8, device="cuda")
    for sizes in ([1, 0, 2], [60, 0, 100]):
        o, od = offs(sizes)
        a = torch.randint(0, 0x7E, (int(o[-1]), K), dtype=torch.uint8, device="cuda")
        sa = torch.randint(120, 130, (K // 512, int(o[-1]), 4), dtype=torch.uint8, device="cuda")
        d = bs.scaled_gemm_grouped_block128(a, sa, b, sb, od, out="f32")
        p = int(o[2])
        f8 = torch.float8_e4m3fn
        w = b[2, N - 256:].view(f8).double() * torch.exp2(
            sb[2][:, N // 128 - 2:].transpose(0, 1).reshape(2, -1).double() - 127).repeat_interleave(128, 0).repeat_interleave(128, 1)
        x = a[p:].view(f8).double() * torch.exp2(
            sa[:, p:].transpose(0, 1).reshape(sizes[2], -1).double() - 127).repeat_interleave(128, 1)
        check(d[p:, N - 256:], from_dev(x @ w.t().contiguous()), from_dev(x.abs() @ w.abs().t().contiguous()), "f32", K,
              f"sizes {sizes}")


def test_dispatch_past_32_bits():
    import torch
    say("quantize_grouped: x past 2^32 bytes")
    M, k = 300000, 8192
    x = torch.randn((M, k), dtype=torch.bfloat16, device="cuda")
    o, od = offs([100, 50])
    index = torch.arange(M - 150, M, dtype=torch.int32, device="cuda")
    got = bs.fp8_quantize_grouped_block128(x, od, "e4m3", index, transposed=True)
    want = bs.fp8_quantize_grouped_block128(x[M - 150:].contiguous(), od, "e4m3", transposed=True)
    assert got[0].equal(want[0]) and got[1].equal(want[1]) and got[2][:, :256].equal(want[2][:, :256]) and got[3][:2].equal(want[3][:2])
