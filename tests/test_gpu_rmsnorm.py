"""The norm to FP8 and its gradient against their float64 references (MI355X).

Errors are counted in u = 2^-24, half a step of FP32.  A sum over k runs through 8 FMAs of a lane, 6
additions across lanes and 6 across pieces of 512 columns: DEPTH = 20 roundings, each at most u of the
sum of magnitudes.
  rstd:  half of (DEPTH + division + eps) u, since the sum of squares has no cancellation, and the
         square root's and the reciprocal's u: (DEPTH / 2 + 1 + 2) u = 13 u;
  y:     rstd and two products: 15 u, and half a step of its type;
  codes: byte for byte those of the FP32 y that the same call returns;
  dx:    g, xh and their difference are rounded once each and the product twice: 5 u (|rstd g| + |rstd xh mean|),
         the mean's own error (DEPTH + 3) u mean|g xh| times |rstd xh|, dh's addition u |dx|;
  dw:    a wave adds at most ceil(rows / 512) rows, and up to 2048 partial sums are added by 16 waves
         (128 each) and then across them: rows / 512 + 1 + 128 + 16 roundings, and xh's own, of sum |dy xh|.
FP16 values below 2^-14 are off by up to 2^-25, half their step; from 65520 on, half a step above its largest
value 65504, FP16 rounds to infinity, so a value within its bound of that or beyond it may be infinite.
"""
import numpy as np
import pytest

import block_scaled_precision_fp8_amd as bs
from gpu_common import from_dev, guarded, say, untouched
from oracle import block128 as b128
from oracle import experts as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DEPTH = 20
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -150, "bf16": 2.0 ** -134, "f16": 2.0 ** -25}
TYPES = ["f32", "bf16", "f16"]


def dtype(t):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[t]


def values(rows, k, t, seed, spread=3):
    import torch
    g = np.random.default_rng(seed)
    x = g.standard_normal((rows, k)) * np.exp2(g.integers(-spread, spread + 1, (rows, 1)))
    x[g.random((rows, k)) < 0.02] *= 20
    x[g.random((rows, k)) < 0.05] = 0
    return torch.from_numpy(x.astype(np.float32)).to(dtype(t)).cuda()


def f64(t):
    return from_dev(t).astype(np.float64)


def close(got, want, bound, t, label):
    """|got - want| <= bound + half a step of type t of the value."""
    got = f64(got)
    over = (t == "f16") & np.isinf(got) & (np.abs(want) + bound >= 65520) & (np.sign(got) == np.sign(want))
    err = np.abs(np.where(over, want, got) - want)
    lim = bound + HALF[t] * (np.abs(want) + bound) + TINY[t]
    worst = float((err / lim).max()) if err.size else 0.0
    say(f"{label}: {worst:.3f} of the bound")
    assert worst <= 1.0, f"{label}: {worst:.3f} of the bound"


def check_norm(x, w, r, y_type, fmt, eps, **kw):
    xt, rt = x.clone(), None if r is None else r.clone()
    got = bs.rmsnorm_quantize_block128(x, w, r, eps=eps, fmt=fmt, y="f32", rstd=True, **kw)
    s = xt.float()
    if rt is not None:
        s = (s + rt.float()).to(rt.dtype)
        import torch
        assert torch.equal(got.h, s)
    y, rstd = ref.rmsnorm(f64(s), None if w is None else f64(w), eps)
    close(got.rstd, rstd, 13 * U * rstd, "f32", "rstd")
    close(got.y, y, 15 * U * np.abs(y), "f32", "y")
    codes, scales = b128.quantize(from_dev(got.y), fmt, 1)
    assert np.array_equal(from_dev(got.codes), codes) and np.array_equal(from_dev(got.scales), scales)
    return got, s


SHAPES = [(1, 1), (1, 128), (3, 40), (5, 513), (16, 8192), (130, 1000), (2, 16384), (3, 20001), (2, 32768), (700, 2048),
          (129, 4096), (1025, 4100)]


@pytest.mark.parametrize("i,shape", enumerate(SHAPES))
def test_norm(i, shape):
    rows, k = shape
    for j in range(4):
        xt, rt, wt = TYPES[(i + j) % 3], (None, "bf16", "f32", "f16")[(i + 2 * j) % 4], (None, "bf16", "f32", "f16")[(i + j) % 4]
        fmt = ("e4m3", "e5m2")[(i + j) % 2]
        say(f"rmsnorm {rows}x{k} x {xt} residual {rt} weight {wt} {fmt}")
        x = values(rows, k, xt, 100 * i + j)
        r = None if rt is None else values(rows, k, rt, 1000 + i)
        w = None if wt is None else values(1, k, wt, 2000 + i, 0)[0].contiguous()
        got, s = check_norm(x, w, r, "f32", fmt, 1e-5)
        for y_type in ("bf16", "f16"):
            # the same FP32 value, rounded once
            y = bs.rmsnorm_quantize_block128(x, w, r, eps=1e-5, fmt=None, y=y_type).y
            assert y.equal(got.y.to(dtype(y_type)))


@pytest.mark.parametrize("off,extra", [(0, 8), (1, 0), (0, 3), (3, 5)])
@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_strides_offsets_and_guards(t, off, extra):
    """Views at odd offsets and row strides, outputs inside canaries."""
    import torch
    rows, k = 37, 1100
    def view(seed):
        v = values(rows, k, t, seed)
        base = torch.zeros(rows * (k + extra) + off + 8, dtype=v.dtype, device="cuda")
        out = base[off:off + rows * (k + extra)].view(rows, k + extra)[:, :k]
        out.copy_(v)
        return out
    say(f"rmsnorm view offset {off} extra {extra} {t}")
    x, r, w = view(1), view(2), values(1, k, t, 3, 0)[0].contiguous()
    want = bs.rmsnorm_quantize_block128(x.contiguous(), w, r.contiguous(), y="f32", rstd=True)
    hb, h = guarded((rows, k), x.dtype, extra_cols=extra + 1, extra_rows=1, tail=16)
    yb, y = guarded((rows, k), torch.float32, extra_cols=extra, extra_rows=1, tail=16)
    sb, rstd = guarded((rows,), torch.float32, tail=16)
    shapes = [tuple(want.codes.shape), tuple(want.scales.shape)]
    bufs = [guarded((int(np.prod(s)),), torch.uint8, tail=64) for s in shapes]
    got = bs.rmsnorm_quantize_block128(x, w, r, y=y, rstd=rstd, h=h, codes=bufs[0][1].view(shapes[0]),
                                       scales=bufs[1][1].view(shapes[1]))
    for a, b in zip(got, want):
        assert a.equal(b)
    assert untouched(hb, (rows, k), extra + 1, 1, 16) and untouched(yb, (rows, k), extra, 1, 16)
    assert untouched(sb, (rows,), tail=16)
    assert all(untouched(b, (int(np.prod(s)),), tail=64) for (b, _), s in zip(bufs, shapes))
    dy, dh = view(4), view(5)
    dx0, dw0 = bs.rmsnorm_backward(dy.contiguous(), want.h, want.rstd, w, dh=dh.contiguous())
    xb, dx = guarded((rows, k), x.dtype, extra_cols=extra, extra_rows=1, tail=16)
    wb, dw = guarded((k,), torch.float32, tail=16)
    size = bs.rmsnorm_backward_workspace(rows, k)
    kb, ws = guarded((size,), torch.uint8, tail=64)
    bs.rmsnorm_backward(dy, h, rstd, w, dh=dh, dx=dx, dweight=dw, workspace=ws)
    assert dx.equal(dx0) and dw.equal(dw0)
    assert untouched(xb, (rows, k), extra, 1, 16) and untouched(wb, (k,), tail=16) and untouched(kb, (size,), tail=64)


def test_in_place():
    """The sum over the residual or over x, y over x, dx over dy, h or dh."""
    x, r, w = values(70, 1500, "bf16", 1), values(70, 1500, "bf16", 2), values(1, 1500, "f32", 3, 0)[0].contiguous()
    say("rmsnorm in place")
    want = bs.rmsnorm_quantize_block128(x, w, r, y="bf16", rstd=True)
    r2 = r.clone()
    got = bs.rmsnorm_quantize_block128(x, w, r2, y="bf16", rstd=True, h=r2)
    assert got.h is r2 and all(a.equal(b) for a, b in zip(got, want))
    x2 = x.clone()
    got = bs.rmsnorm_quantize_block128(x2, w, r, y="bf16", rstd=True, h=x2)
    assert got.h is x2 and all(a.equal(b) for a, b in zip(got, want))
    x2 = x.clone()
    assert bs.rmsnorm_quantize_block128(x2, w, y=x2).y.equal(bs.rmsnorm_quantize_block128(x, w, y="bf16").y)
    dy, dh = values(70, 1500, "bf16", 4), values(70, 1500, "bf16", 5)
    dx, dw = bs.rmsnorm_backward(dy, want.h, want.rstd, w, dh=dh)
    for i in range(3):
        t = [dy.clone(), want.h.clone(), dh.clone()]
        a, b = bs.rmsnorm_backward(t[0], t[1], want.rstd, w, dh=t[2], dx=t[i])
        assert a is t[i] and a.equal(dx) and b.equal(dw)


def test_not_finite_and_zero_rows():
    """A NaN takes its row, an infinity is NaN in a row of zeros, a row of zeros without eps is NaN; blocks
    with any of them hold the NaN scale and NaN codes, and other rows nothing of it."""
    import torch
    say("rmsnorm of non-finite values")
    x = values(9, 700, "f32", 7)
    x[x == 0] = 1.0
    clean = bs.rmsnorm_quantize_block128(x, y="f32", eps=0.0)
    x[1, 300], x[3, 5], x[5], x[7, 699] = float("nan"), float("inf"), 0.0, -float("inf")
    got = bs.rmsnorm_quantize_block128(x, y="f32", eps=0.0, rstd=True)
    y = from_dev(got.y)
    assert np.isnan(y[1]).all() and np.isnan(y[5]).all()
    for row, col in ((3, 5), (7, 699)):
        assert np.isnan(y[row, col]) and not np.delete(y[row], col).any() and from_dev(got.rstd)[row] == 0
    codes, scales = b128.quantize(y, "e4m3", 1)
    assert np.array_equal(from_dev(got.codes), codes) and np.array_equal(from_dev(got.scales), scales)
    for row in (0, 2, 4, 6, 8):
        assert got.y[row].equal(clean.y[row]) and got.codes[row].equal(clean.codes[row])
    dy = values(9, 700, "f32", 8)
    dx, _ = bs.rmsnorm_backward(dy, x, got.rstd)
    ok, _ = bs.rmsnorm_backward(dy[[0, 2, 4, 6, 8]], x[[0, 2, 4, 6, 8]], got.rstd[[0, 2, 4, 6, 8]].contiguous())
    assert dx[[0, 2, 4, 6, 8]].equal(ok) and torch.isnan(dx[1]).all()


@pytest.mark.parametrize("i,shape", enumerate(SHAPES + [(3000, 600), (6000, 130)]))
def test_backward(i, shape):
    rows, k = shape
    for j in range(3):
        yt, ht = TYPES[(i + j) % 3], TYPES[(i + 2 * j) % 3]
        at, wt = (None, "bf16", "f32", "f16")[(i + j) % 4], (None, "bf16", "f32", "f16")[(i + 3 * j) % 4]
        say(f"rmsnorm_backward {rows}x{k} dy {yt} h {ht} dh {at} weight {wt}")
        dy, h = values(rows, k, yt, 50 * i + j), values(rows, k, ht, 3000 + i)
        dh = None if at is None else values(rows, k, at, 4000 + i)
        w = None if wt is None else values(1, k, wt, 5000 + i, 0)[0].contiguous()
        rstd = bs.rmsnorm_quantize_block128(h, y="f32", rstd=True).rstd
        start = values(1, k, "f32", 6000)[0].contiguous()
        dx, dw = bs.rmsnorm_backward(dy, h, rstd, w, dh=dh)
        more = start.clone()
        bs.rmsnorm_backward(dy, h, rstd, w, dh=dh, dweight=more, accumulate=True)
        alone, none = bs.rmsnorm_backward(dy, h, rstd, w, dh=dh, weight_grad=False)
        edx, edw, (sg, sm, sw) = ref.rmsnorm_backward(f64(dy), f64(h), f64(rstd), None if w is None else f64(w),
                                                      None if dh is None else f64(dh))
        xh = np.abs(f64(h) * f64(rstd)[:, None])
        g = np.abs(f64(dy) * (1.0 if w is None else f64(w)))
        means = np.abs(f64(rstd))[:, None] * xh * (g * xh).mean(1, keepdims=True)
        close(dx, edx, 5 * U * (sg + sm) + (DEPTH + 3) * U * means + U * np.abs(edx), ht, "dx")
        depth = (rows / 512 + 1 + 128 + 16 + 2) * U
        close(dw, edw, depth * sw, "f32", "dw")
        assert more.equal(start + dw) and none is None and alone.equal(dx)


def test_no_rows():
    import torch
    x = torch.zeros((0, 300), device="cuda")
    got = bs.rmsnorm_quantize_block128(x, y="bf16", rstd=True)
    assert got.codes.shape == (0, 320) and got.y.shape == (0, 300) and got.rstd.shape == (0,)
    start = values(1, 300, "f32", 1)[0].contiguous()
    dw = start.clone()
    assert bs.rmsnorm_backward(x, x, got.rstd, dweight=dw, accumulate=True)[0].shape == (0, 300) and dw.equal(start)
    bs.rmsnorm_backward(x, x, got.rstd, dweight=dw)
    assert not dw.any()
    assert bs.rmsnorm_quantize_block128(torch.zeros((3, 0), device="cuda")).codes.shape == (3, 0)


def test_refusals_launch_nothing():
    import torch
    x, w = values(4, 64, "bf16", 1), values(1, 64, "f32", 2)[0].contiguous()
    y = torch.full((4, 64), 7.0, device="cuda")
    r = torch.ones(4, device="cuda")
    bad = [lambda: bs.rmsnorm_quantize_block128(x.double(), y=y),
           lambda: bs.rmsnorm_quantize_block128(x[0], y=y),
           lambda: bs.rmsnorm_quantize_block128(x.t(), y=y),
           lambda: bs.rmsnorm_quantize_block128(x, w[:63], y=y),
           lambda: bs.rmsnorm_quantize_block128(x, w[None], y=y),
           lambda: bs.rmsnorm_quantize_block128(x, w, x[:3], y=y),
           lambda: bs.rmsnorm_quantize_block128(x, w, x.cpu(), y=y),
           lambda: bs.rmsnorm_quantize_block128(x, w, x, y=y, h=y),
           lambda: bs.rmsnorm_quantize_block128(x, w, y=y, h=x),
           lambda: bs.rmsnorm_quantize_block128(x, w, y=y[:3]),
           lambda: bs.rmsnorm_quantize_block128(x, w, y="f64"),
           lambda: bs.rmsnorm_quantize_block128(x, w, y=y, fmt="e3m4"),
           lambda: bs.rmsnorm_quantize_block128(x, w, fmt=None),
           lambda: bs.rmsnorm_quantize_block128(x, w, y=y, fmt=None, codes=x),
           lambda: bs.rmsnorm_quantize_block128(x, w, y=y, rstd=r[:3]),
           lambda: bs.rmsnorm_quantize_block128(x, w, y=y, codes=torch.zeros((4, 32), dtype=torch.uint8, device="cuda")),
           lambda: bs.rmsnorm_quantize_block128(x.expand(4, 64)[:1].expand(4, 64), w, y=y),
           lambda: bs.rmsnorm_backward(x, y, r[:3]), lambda: bs.rmsnorm_backward(x, y[:3], r),
           lambda: bs.rmsnorm_backward(x, y, r, w, dh=x[:, :32]), lambda: bs.rmsnorm_backward(x, y, r, w, dx=x),
           lambda: bs.rmsnorm_backward(x, y, r, w, accumulate=True),
           lambda: bs.rmsnorm_backward(x, y, r, w, weight_grad=False, dweight=w),
           lambda: bs.rmsnorm_backward(x, y, r, w, dweight=w[:32]),
           lambda: bs.rmsnorm_backward(x, y, r, w, workspace=torch.zeros(8, dtype=torch.uint8, device="cuda"))]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            print(i)
    with pytest.raises(RuntimeError, match="INVALID"):
        bs.rmsnorm_quantize_block128(x, w, y=y, eps=-1.0)
    with pytest.raises(RuntimeError, match="UNSUPPORTED"):
        bs.rmsnorm_quantize_block128(torch.zeros((1, 32800), device="cuda"))
    assert bool((y == 7.0).all())


def test_streams_and_graph():
    """Calls on two streams at once, and a captured forward and backward pass replayed on new inputs with
    an autograd graph of the same tensors alive."""
    import torch
    say("rmsnorm on two streams")
    xs = [values(n, 3000, "bf16", n) for n in (3, 500, 1500)]
    w = values(1, 3000, "f32", 9, 0)[0].contiguous()

    def step(x):
        f = bs.rmsnorm_quantize_block128(x, w, rstd=True, y="bf16")
        return [f.codes, f.scales, f.y, *bs.rmsnorm_backward(f.y, x, f.rstd, w)]

    want = [step(x) for x in xs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for i in range(12):
        with torch.cuda.stream(streams[i % 2]):
            got.append(step(xs[i % 3]))
    torch.cuda.synchronize()
    assert all(a.equal(b) for i, g in enumerate(got) for a, b in zip(g, want[i % 3]))
    say("rmsnorm in a graph")
    leaf = w.clone().requires_grad_()
    alive = (xs[1].float() * leaf).sum()
    x, side = xs[1].clone(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(x)
    for i in range(3):
        x.copy_(values(500, 3000, "bf16", 40 + i))
        graph.replay()
        assert all(a.equal(b) for a, b in zip(out, step(x)))
    alive.backward()
    assert leaf.grad is not None


def test_versions_count_what_is_written():
    import torch
    x, r = values(4, 64, "f32", 1), values(4, 64, "f32", 2)
    y = torch.empty_like(x)
    before = [t._version for t in (r, y)]
    bs.rmsnorm_quantize_block128(x, residual=r, h=r, y=y)
    assert [t._version for t in (r, y)] == [b + 1 for b in before]
    w = torch.ones(64, device="cuda", requires_grad=True)
    dw = torch.zeros(64, device="cuda")
    v = dw._version
    bs.rmsnorm_backward(x, r, torch.ones(4, device="cuda"), w.detach(), dweight=dw)
    assert dw._version == v + 1


@pytest.mark.parametrize("k", [100, 700, 1500, 2600, 5000, 9000, 20001])
def test_a_row_is_the_same_in_every_call(k):
    """Forward results and dx of a row do not depend on the rows around it or on their number."""
    say(f"rmsnorm: rows alone and among others, k {k}")
    x, dy, w = values(600, k, "bf16", 1), values(600, k, "f32", 2), values(1, k, "f32", 3, 0)[0].contiguous()
    f = bs.rmsnorm_quantize_block128(x, w, y="f32", rstd=True)
    dx, _ = bs.rmsnorm_backward(dy, x, f.rstd, w)
    for part in (slice(0, 1), slice(5, 8), slice(100, 500)):
        g = bs.rmsnorm_quantize_block128(x[part], w, y="f32", rstd=True)
        assert g.rstd.equal(f.rstd[part]) and g.y.equal(f.y[part]) and g.codes.equal(f.codes[part])
        assert bs.rmsnorm_backward(dy[part], x[part], g.rstd, w)[0].equal(dx[part])


def test_rows_past_32_bits():
    import torch
    rows, k = 280000, 8192
    say("rmsnorm of more than 2^32 bytes")
    x = torch.randn((rows, k), dtype=torch.bfloat16, device="cuda")
    got = bs.rmsnorm_quantize_block128(x, y="bf16", rstd=True)
    dx, dw = bs.rmsnorm_backward(got.y, x, got.rstd)
    last = slice(rows - 40, rows)
    want = bs.rmsnorm_quantize_block128(x[last].contiguous(), y="bf16", rstd=True)
    assert got.y[last].equal(want.y) and got.codes[last].equal(want.codes) and got.rstd[last].equal(want.rstd)
    assert got.scales[:, last].equal(want.scales)
    assert dx[last].equal(bs.rmsnorm_backward(want.y, x[last].contiguous(), want.rstd)[0])
    assert bool(torch.isfinite(dw).all())
