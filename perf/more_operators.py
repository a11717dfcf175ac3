"""Cases of the norm and of the grouped block-of-128 FP8 operators, with their plain forms.

Five operators of a step of a network with experts:

  norm        the residual's addition and root-mean-square norm, to FP8 codes with one
              power-of-two (E8M0) scale per 1 x 128 block, and to 16 or 32 bits
  norm_grad   its gradients of the input and of the weight
  dispatch    FP8 quantisation of rows sorted by expert: taken by an index, by rows and
              transposed, each group's columns of the transpose padded to blocks of 128
  grouped     D[i] = A[i] B[e]^T, e the expert of row i: forward products and, with
              transposed weights, gradients of the input
  weight_grad D[e] = sum of A[:, i] B[:, i]^T over the rows i of expert e (+ C[e])

With ``own`` false, ``run`` computes them from elementary torch operations; with it
true, through the package's entry points.
"""
import math
import random

import torch

own = False

FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"none": 0, "f32": 4, "bf16": 2, "f16": 2}
DEV = "cuda"


# ----------------------------------------------------------------------------------------
# Cases
# ----------------------------------------------------------------------------------------
def listed():
    n = dict(op="norm", eps=1e-6, fmt="e4m3", w_type="bf16")
    b = dict(op="norm_grad", eps=1e-6, w_type="bf16")
    q = dict(op="dispatch")
    g = dict(op="grouped", alpha=1.0, accumulate=False)
    w = dict(op="weight_grad")
    return [
        # 16 decoded tokens, ahead of a projection, the residual updated in place: latency
        dict(n, name="norm_16x8192", rows=16, k=8192, x_type="bf16", h_type="bf16", y_type="none", statistics=False),
        # a training batch: codes for the dense products, y for the experts' dispatch, the
        # statistics for the backward pass
        dict(n, name="norm_16384x4096", rows=16384, k=4096, x_type="bf16", h_type="bf16", y_type="bf16",
             statistics=True),
        # its gradient, with the one that comes along the residual
        dict(b, name="norm_grad_16384x4096", rows=16384, k=4096, dy_type="bf16", h_type="bf16", dh_type="bf16"),
        # odd sizes, FP32, without a residual
        dict(b, name="norm_grad_777x5001", rows=777, k=5001, dy_type="f32", h_type="f32", dh_type="none"),
        # 8192 tokens, two experts each out of 8: rows for the forward product, the transpose
        # for the weight gradient
        dict(q, name="dispatch_16384x4096", rows=16384, groups=8, spread=0.5, k=4096, type="bf16", fmt="e4m3",
             index=True, want="both"),
        # gradients of an odd number of rows over many experts, some without any
        dict(q, name="dispatch_grad_1111x4001", rows=1111, groups=64, spread=1.5, k=4001, type="bf16", fmt="e5m2",
             index=False, want="both"),
        # one decoded token sent to 8 of 16 experts: the smallest call
        dict(g, name="grouped_8x1024x4096", rows=8, groups=16, spread=3.0, N=1024, K=4096, a_fmt="e4m3",
             b_fmt="e4m3", b_block_rows=128, out="bf16"),
        # 32 decoded tokens, four experts each out of 64: streams most of the weights
        dict(g, name="grouped_128x2048x4096", rows=128, groups=64, spread=0.7, N=2048, K=4096, a_fmt="e4m3",
             b_fmt="e4m3", b_block_rows=128, out="bf16"),
        # a prompt of odd length, two experts each out of 16, partial tiles and K blocks
        dict(g, name="grouped_2222x4000x4064", rows=2222, groups=16, spread=0.7, N=4000, K=4064, a_fmt="e4m3",
             b_fmt="e4m3", b_block_rows=128, out="bf16"),
        # the feed-forward product of a training batch over 8 experts
        dict(g, name="grouped_16384x14336x4096", rows=16384, groups=8, spread=0.5, N=14336, K=4096, a_fmt="e4m3",
             b_fmt="e4m3", b_block_rows=128, out="bf16"),
        # weight gradients of 8 experts, added to the FP32 gradients
        dict(w, name="weight_grad_16384x4096x4096", rows=16384, groups=8, spread=0.5, m=4096, n=4096, a_fmt="e5m2",
             b_fmt="e4m3", out="f32", accumulate=True),
        # those of many small experts, of odd sizes, some without rows
        dict(w, name="weight_grad_2222x1000x2001", rows=2222, groups=32, spread=1.5, m=1000, n=2001, a_fmt="e5m2",
             b_fmt="e4m3", out="bf16", accumulate=False),
    ]


def _size(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("norm", "norm_grad", "dispatch", "grouped", "weight_grad"))
    pick = rng.choice
    rows, groups = _size(rng, 1, 16384), _size(rng, 1, 256)
    ragged = dict(op=op, rows=rows, groups=groups, spread=pick((0.0, 0.5, 1.5)))
    fmts = dict(a_fmt=pick(("e4m3", "e5m2")), b_fmt=pick(("e4m3", "e5m2")), out=pick(("f32", "bf16", "bf16", "f16")),
                accumulate=pick((False, True)))
    if op == "norm":
        return dict(op=op, rows=rows, k=_size(rng, 16, 4096), x_type=pick(("f32", "bf16", "f16")),
                    h_type=pick(("none", "f32", "bf16", "f16")), w_type=pick(("none", "f32", "bf16")),
                    y_type=pick(("none", "bf16", "f32")), statistics=pick((False, True)), eps=pick((1e-6, 1e-5)),
                    fmt=pick(("e4m3", "e5m2")))
    if op == "norm_grad":
        return dict(op=op, rows=rows, k=_size(rng, 16, 4096), dy_type=pick(("f32", "bf16", "f16")),
                    h_type=pick(("f32", "bf16", "f16")), dh_type=pick(("none", "f32", "bf16")),
                    w_type=pick(("none", "f32", "bf16")), eps=1e-6)
    if op == "dispatch":
        return dict(ragged, k=_size(rng, 1, 4096), type=pick(("f32", "bf16", "f16")), fmt=pick(("e4m3", "e5m2")),
                    index=pick((False, True)), want=pick(("rows", "transposed", "both")))
    if op == "grouped":
        K = 32 * _size(rng, 1, 128)
        return dict(ragged, K=K, N=_size(rng, 1, min(14336, (1 << 28) // (groups * K))), alpha=pick((1.0, 0.5)),
                    b_block_rows=pick((1, 128, 128)), **fmts)
    m = _size(rng, 1, 4096)
    return dict(ragged, m=m, n=_size(rng, 1, min(4096, (1 << 26) // (groups * m) + 1)), **fmts)


def _up(a, b):
    return (a + b - 1) // b * b


def _sizes(case):
    """The groups' sizes: rows given to groups whose shares are log-normal of the case's spread."""
    rng = random.Random("%d %d %g" % (case["rows"], case["groups"], case["spread"]))
    shares = [math.exp(rng.gauss(0.0, case["spread"])) for _ in range(case["groups"])]
    got = [0] * case["groups"]
    for e in rng.choices(range(case["groups"]), shares, k=case["rows"]):
        got[e] += 1
    if case["rows"] <= case["groups"]:            # a token's experts are different ones
        first = sorted(range(case["groups"]), key=lambda e: -shares[e])[:case["rows"]]
        got = [int(e in first) for e in range(case["groups"])]
    return got


def work(case):
    op = case["op"]
    if op == "norm":
        n = case["rows"] * case["k"]
        each = SIZE[case["x_type"]] + 2 * SIZE[case["h_type"]] + 1 + SIZE[case["y_type"]]
        return {"bytes": n * each + n // 128 + case["k"] * SIZE[case["w_type"]] + 4 * case["rows"] * case["statistics"],
                "flops": 0}
    if op == "norm_grad":
        each = SIZE[case["dy_type"]] + 2 * SIZE[case["h_type"]] + SIZE[case["dh_type"]]
        return {"bytes": case["rows"] * case["k"] * each + case["k"] * (4 + SIZE[case["w_type"]]) + 4 * case["rows"],
                "flops": 0}
    sizes = _sizes(case)
    rows, total = case["rows"], sum(_up(s, 128) for s in sizes)
    if op == "dispatch":
        k = case["k"]
        source = (rows + 1) // 2 if case["index"] else rows
        n = source * k * SIZE[case["type"]]
        n += rows * (_up(k, 32) + k // 128) if case["want"] != "transposed" else 0
        n += k * (total + total // 128) if case["want"] != "rows" else 0
        return {"bytes": n, "flops": 0}
    out = SIZE[case["out"]] * (2 if case["accumulate"] else 1)
    if op == "grouped":
        N, K, used = case["N"], case["K"], sum(s > 0 for s in sizes)
        return {"bytes": (rows + used * N) * K + rows * N * out, "flops": 2 * rows * N * K}
    m, n = case["m"], case["n"]
    return {"bytes": rows * (m + n) + case["groups"] * m * n * out, "flops": 2 * rows * m * n}


# ----------------------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------------------
def _normal(gen, shape, std):
    return torch.randn(shape, generator=gen, device=DEV) * std


def _laplace(gen, shape, scale):
    u = torch.rand(shape, generator=gen, device=DEV) - 0.5
    return -scale * torch.sign(u) * torch.log1p(-2 * u.abs() * (1 - 2.0 ** -20))


def _activations(gen, rows, k):
    """N(0, 1) with one entry in a thousand thirty times larger."""
    x = _normal(gen, (rows, k), 1.0)
    far = torch.rand((rows, k), generator=gen, device=DEV) < 0.001
    return torch.where(far, x * 30, x)


def _operand(gen, rows, k, fmt):
    return _laplace(gen, (rows, k), 1e-3) if fmt == "e5m2" else _activations(gen, rows, k)


def _ragged(case, seed):
    """The groups' sizes in an order of the seed's own, their offsets on the host and on the device."""
    sizes = _sizes(case)
    random.Random(seed).shuffle(sizes)
    offsets = [0]
    for s in sizes:
        offsets.append(offsets[-1] + s)
    return dict(sizes=sizes, total=sum(_up(s, 128) for s in sizes), words=sum(_up(s, 512) // 512 for s in sizes),
                offsets=torch.tensor(offsets, dtype=torch.int32, device=DEV))


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op = case["op"]
    if op in ("norm", "norm_grad"):
        rows, k = case["rows"], case["k"]
        s = dict(case, weight=None)
        if case["w_type"] != "none":
            s["weight"] = (1 + _normal(gen, (k,), 0.2)).to(TYPES[case["w_type"]])
        if op == "norm":
            s["x"] = _activations(gen, rows, k).to(TYPES[case["x_type"]])
            s["residual"] = None
            if case["h_type"] != "none":
                s["residual"] = _normal(gen, (rows, k), 2.0).to(TYPES[case["h_type"]])
                s["h"] = torch.empty_like(s["residual"])
            return s
        s["dy"] = _laplace(gen, (rows, k), 1e-3).to(TYPES[case["dy_type"]])
        s["h"] = (_activations(gen, rows, k) * 2).to(TYPES[case["h_type"]])
        s["rstd"] = torch.rsqrt(s["h"].float().square().mean(1) + case["eps"])
        s["dh"] = None
        if case["dh_type"] != "none":
            s["dh"] = _laplace(gen, (rows, k), 1e-3).to(TYPES[case["dh_type"]])
        return s
    s = dict(case, **_ragged(case, seed))
    rows = case["rows"]
    if op == "dispatch":
        source = (rows + 1) // 2 if case["index"] else rows       # two experts a token
        s["x"] = _operand(gen, source, case["k"], case["fmt"]).to(TYPES[case["type"]])
        s["index"] = None
        if case["index"]:
            s["index"] = (torch.randperm(rows, generator=gen, device=DEV) // 2).to(torch.int32)
        return s
    s["d"] = None
    if op == "grouped":
        N, K, E, br = case["N"], case["K"], case["groups"], case["b_block_rows"]
        s["a"], s["sa"] = _quantize(_operand(gen, rows, K, case["a_fmt"]), case["a_fmt"], 1)
        s["b"] = torch.empty((E, N, K), dtype=torch.uint8, device=DEV)
        s["sb"] = torch.empty((E, (K + 511) // 512, (N + br - 1) // br, 4), dtype=torch.uint8, device=DEV)
        for e in range(E):
            s["b"][e], s["sb"][e] = _quantize(_normal(gen, (N, K), 1.0 if br == 1 else 0.02), case["b_fmt"], br)
        if case["accumulate"]:
            s["d"] = _normal(gen, (rows, N), 1e-2).to(TYPES[case["out"]])
        return s
    for x, w in (("a", case["m"]), ("b", case["n"])):
        v = _operand(gen, rows, w, case[x + "_fmt"])
        codes, scales = _quantize_columns(v, s, case[x + "_fmt"])
        # the buffers as a program allocates them, for any sizes of as many groups
        most = _up(rows + 127 * min(case["groups"], rows), 128)
        s[x] = torch.zeros((w, most), dtype=torch.uint8, device=DEV)
        s[x][:, :s["total"]] = codes
        s["s" + x] = torch.full((rows // 512 + min(case["groups"], rows), w, 4), 127, dtype=torch.uint8, device=DEV)
        s["s" + x][:s["words"]] = scales
    if case["accumulate"]:
        s["d"] = _normal(gen, (case["groups"], case["m"], case["n"]), 1e-2).to(TYPES[case["out"]])
    return s


# ----------------------------------------------------------------------------------------
# Plain forms
# ----------------------------------------------------------------------------------------
#: The formats' largest finite value, as a fraction of the power of two above it.
TOP = {"e4m3": (0.875, 9), "e5m2": (0.875, 16)}


def _exponents(amax, fmt):
    """The smallest e with F 2^e >= amax, in [-127, 127]; 0 where amax is 0."""
    frac, above = TOP[fmt]
    m, e = torch.frexp(amax)
    e = e.to(torch.int32) - above + (m > frac).to(torch.int32)
    return torch.where(amax == 0, 0, e.clamp(-127, 127))


def _power(e):
    """2^e in FP32, exactly, for e in [-126, 127]."""
    return ((e + 127) << 23).view(torch.float32)


def _blocks(x, fmt, block_rows):
    """Codes (rows x k up to a multiple of 32, zeros past k) and the exponents of the blocks of x."""
    rows, k = x.shape
    R, Kb = (rows + block_rows - 1) // block_rows, (k + 127) // 128
    xp = torch.nn.functional.pad(x.float(), (0, 128 * Kb - k, 0, R * block_rows - rows))
    xb = xp.view(R, block_rows, Kb, 128)
    e = _exponents(xb.abs().amax((1, 3)), fmt)
    y = (xb * _power(-e)[:, None, :, None]).view(R * block_rows, Kb * 128)
    return y[:rows, :_up(k, 32)].to(FP8[fmt]).view(torch.uint8).contiguous(), e


def _quantize(x, fmt, block_rows):
    """Codes and E8M0 scales [K / 512][rows of blocks][4]: byte (g, r, j) is K block 4 g + j's."""
    codes, e = _blocks(x, fmt, block_rows)
    R, Kb = e.shape
    scales = torch.full((R, _up(Kb, 4)), 127, dtype=torch.uint8, device=x.device)
    scales[:, :Kb] = (e + 127).to(torch.uint8)
    return codes, scales.view(R, -1, 4).transpose(0, 1).contiguous()


def _dequantize(codes, scales, fmt, block_rows):
    rows, K = codes.shape
    s = scales.transpose(0, 1).reshape(scales.shape[1], -1).view(torch.float8_e8m0fnu).float()
    s = s.repeat_interleave(block_rows, 0)[:rows].repeat_interleave(128, 1)[:, :K]
    return codes.view(FP8[fmt]).float() * s


def _layout(s):
    """Of each block of 128 columns of a transpose in groups: its word of scales and its byte in it;
    and each group's first block."""
    sizes = s["offsets"].diff().long()
    blocks, words = (sizes + 127) // 128, (sizes + 511) // 512
    first = blocks.cumsum(0) - blocks
    e = torch.arange(len(s["sizes"]), device=DEV).repeat_interleave(blocks, output_size=s["total"] // 128)
    j = torch.arange(s["total"] // 128, device=DEV) - first[e]
    return (words.cumsum(0) - words)[e] + j // 4, j % 4, first


def _quantize_columns(x, s, fmt):
    """Codes and scales of the transpose of x, rows of a group to columns from a multiple of 128 on."""
    word, byte, first = _layout(s)
    starts = s["offsets"].long()
    i = torch.arange(x.shape[0], device=DEV)
    e = torch.searchsorted(starts, i, right=True) - 1
    xp = torch.zeros((s["total"], x.shape[1]), device=DEV)
    xp[first[e] * 128 + i - starts[e]] = x.float()
    codes, ex = _blocks(xp.t(), fmt, 1)
    scales = torch.full((s["words"], x.shape[1], 4), 127, dtype=torch.uint8, device=DEV)
    scales[word, :, byte] = (ex + 127).to(torch.uint8).t()
    return codes, scales


def _dequantize_columns(codes, scales, s, fmt):
    word, byte, _ = _layout(s)
    f = scales[word, :, byte].view(torch.float8_e8m0fnu).float().t()
    return codes[:, :s["total"]].view(FP8[fmt]).float() * f.repeat_interleave(128, 1)


def _ends(sizes, step=1):
    """(group, first, end) of the groups that have rows, their sizes rounded up to step."""
    got, at = [], 0
    for e, n in enumerate(sizes):
        if n:
            got.append((e, at, at + _up(n, step)))
        at += _up(n, step)
    return got


def _norm_plain(s):
    x, w = s["x"].float(), s["weight"]
    h = x
    if s["residual"] is not None:
        h = s["h"].copy_(x + s["residual"].float()).float()
    rstd = torch.rsqrt(h.square().mean(1) + s["eps"])
    y = h * rstd[:, None]
    if w is not None:
        y = y * w.float()
    codes, scales = _quantize(y, s["fmt"], 1)
    return (codes, scales, None if s["y_type"] == "none" else y.to(TYPES[s["y_type"]]),
            None if s["residual"] is None else s["h"], rstd if s["statistics"] else None)


def _norm_grad_plain(s):
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xh = s["h"].float() * rstd
    g = dy if s["weight"] is None else dy * s["weight"].float()
    dx = rstd * (g - xh * (g * xh).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return dx.to(s["h"].dtype), (dy * xh).sum(0)


def _grouped_plain(s):
    a = _dequantize(s["a"], s["sa"], s["a_fmt"], 1)
    d = torch.cat([a[i:j] @ _dequantize(s["b"][e], s["sb"][e], s["b_fmt"], s["b_block_rows"]).t()
                   for e, i, j in _ends(s["sizes"])])
    d = s["alpha"] * d
    if s["accumulate"]:
        return s["d"].copy_(d + s["d"].float())
    return d.to(TYPES[s["out"]])


def _weight_grad_plain(s):
    a = _dequantize_columns(s["a"], s["sa"], s, s["a_fmt"])
    b = _dequantize_columns(s["b"], s["sb"], s, s["b_fmt"])
    d = torch.zeros((s["groups"], s["m"], s["n"]), device=DEV)
    [torch.mm(a[:, i:j], b[:, i:j].t(), out=d[e]) for e, i, j in _ends(s["sizes"], 128)]
    if s["accumulate"]:
        return s["d"].copy_(d + s["d"].float())
    return d.to(TYPES[s["out"]])


def _as_values(codes, scales, fmt):
    """Codes and scale bytes as the values that they stand for."""
    return [codes.view(FP8[fmt]), scales.view(torch.float8_e8m0fnu)]


def run(state):
    s, op = state, state["op"]
    if own:
        import block_scaled_precision_fp8_amd as bs
    if op == "norm":
        if own:
            got = bs.rmsnorm_quantize_block128(
                s["x"], s["weight"], s["residual"], eps=s["eps"], fmt=s["fmt"],
                y=None if s["y_type"] == "none" else s["y_type"], rstd=s["statistics"],
                h=None if s["residual"] is None else s["h"])
        else:
            got = _norm_plain(s)
        return _as_values(got[0], got[1], s["fmt"]) + [t for t in got[2:] if t is not None]
    if op == "norm_grad":
        if own:
            return bs.rmsnorm_backward(s["dy"], s["h"], s["rstd"], s["weight"], dh=s["dh"])
        return _norm_grad_plain(s)
    if op == "dispatch":
        rows, columns = s["want"] != "transposed", s["want"] != "rows"
        if own:
            got = bs.fp8_quantize_grouped_block128(s["x"], s["offsets"], s["fmt"], index=s["index"], rows=rows,
                                                   transposed=columns)
            if columns:                           # what the groups hold of the buffers for any sizes
                got = got[:-2] + (got[-2][:, :s["total"]], got[-1][:s["words"]])
        else:
            x = s["x"] if s["index"] is None else s["x"][s["index"].long()]
            got = _quantize(x, s["fmt"], 1) if rows else ()
            got += _quantize_columns(x, s, s["fmt"]) if columns else ()
        return [_as_values(got[i], got[i + 1], s["fmt"]) for i in range(0, len(got), 2)]
    if op == "grouped":
        if own:
            return bs.scaled_gemm_grouped_block128(
                s["a"], s["sa"], s["b"], s["sb"], s["offsets"], s["a_fmt"], s["b_fmt"], s["b_block_rows"],
                out=s["out"], alpha=s["alpha"], c=s["d"], beta=1.0 if s["accumulate"] else 0.0, d=s["d"])
        return _grouped_plain(s)
    if own:
        return bs.scaled_gemm_grouped_wgrad_block128(
            s["a"], s["sa"], s["b"], s["sb"], s["offsets"], s["a_fmt"], s["b_fmt"], out=s["out"], c=s["d"],
            beta=1.0 if s["accumulate"] else 0.0, d=s["d"])
    return _weight_grad_plain(s)


# ----------------------------------------------------------------------------------------
# The same from the definitions, in 64 bits
# ----------------------------------------------------------------------------------------
def _grid(fmt):
    """The finite non-negative values of a format, by code."""
    bias, man, top = (7, 3, 0x7E) if fmt == "e4m3" else (15, 2, 0x7B)
    parts = [divmod(c, 2 ** man) for c in range(top + 1)]
    return torch.tensor([math.ldexp(f + (2 ** man if e else 0), max(e, 1) - bias - man) for e, f in parts],
                        dtype=torch.float64, device=DEV)


def _two_to(e):
    """2^e in 64 bits, from a table of the exact powers."""
    return torch.tensor([math.ldexp(1.0, i) for i in range(-400, 401)], dtype=torch.float64, device=DEV)[e.long() + 400]


def _exact_row(x, fmt):
    """The values of the codes of the rows of x (its width up to a multiple of 32) and its scales by block."""
    k, top, grid = x.shape[1], _grid(fmt)[-1], _grid(fmt)
    amax = torch.stack([c.abs().amax(1) for c in x.split(128, 1)], 1)
    s = _two_to(torch.ceil(torch.log2(amax / top)).clamp(-127, 127))
    s = torch.where((s / 2 * top >= amax) & (s > 2.0 ** -127), s / 2, s)
    s = torch.where(s * top < amax, s * 2, s)
    s = torch.where(amax == 0, 1.0, s)
    y = (x / s.repeat_interleave(128, 1)[:, :k]).abs().contiguous()
    hi = torch.searchsorted(grid, y).clamp(max=grid.numel() - 1)
    lo = (hi - 1).clamp(min=0)
    below, above = y - grid[lo], grid[hi] - y
    near = grid[torch.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)]
    return torch.nn.functional.pad(torch.copysign(near, x), (0, _up(k, 32) - k)), s


def _exact_rows(x, fmt):
    """The same for many rows, some at a time, with the scales in words of four."""
    parts = [_exact_row(x[r:r + 2048], fmt) for r in range(0, x.shape[0], 2048)]
    s = torch.cat([p[1] for p in parts])
    s = torch.nn.functional.pad(s, (0, _up(s.shape[1], 4) - s.shape[1]), value=1.0)
    return [torch.cat([p[0] for p in parts]), s.view(s.shape[0], -1, 4).transpose(0, 1)]


def _exact_columns(x, sizes, fmt):
    """Group by group: codes of the transpose, zeros up to a multiple of 128, and whole words of scales."""
    codes, scales = [], []
    for part in x.split(sizes):
        if part.shape[0]:
            c, s = _exact_rows(part.t(), fmt)
            codes.append(torch.nn.functional.pad(c, (0, _up(c.shape[1], 128) - c.shape[1])))
            scales.append(s)
    return [torch.cat(codes, 1), torch.cat(scales)]


def _signed(codes, fmt):
    c = codes.long()
    v = _grid(fmt)[c & 127]
    return torch.where(c >= 128, -v, v)


def _exact_operand(codes, scales, fmt, block_rows=1):
    rows, K = codes.shape
    ri, ki = torch.arange(rows, device=DEV) // block_rows, torch.arange(K, device=DEV) // 128
    return _signed(codes, fmt) * _two_to(scales.long() - 127)[ki // 4, :, ki % 4].t()[ri]


def _exact_norm(s):
    x, w = s["x"].double(), s["weight"]
    h = x if s["residual"] is None else (x + s["residual"].double()).to(s["residual"].dtype).double()
    rstd = 1 / torch.sqrt((h * h).sum(1) / s["k"] + s["eps"])
    y = h * rstd[:, None] * (1.0 if w is None else w.double())
    more = ([] if s["y_type"] == "none" else [y]) + ([] if s["residual"] is None else [h])
    return _exact_rows(y, s["fmt"]) + more + ([rstd] if s["statistics"] else [])


def _exact_norm_grad(s):
    dy, h, r = s["dy"].double(), s["h"].double(), s["rstd"].double()[:, None]
    g = dy * (1.0 if s["weight"] is None else s["weight"].double())
    dx = r * g - h * r ** 3 * ((g * h).sum(1, keepdim=True) / s["k"])
    return dx if s["dh"] is None else dx + s["dh"].double(), (dy * h * r).sum(0)


def exact(case, seed):
    s = prepare(case, seed)
    op, d = case["op"], s.get("d")
    if op == "norm":
        return _exact_norm(s)
    if op == "norm_grad":
        return _exact_norm_grad(s)
    if op == "dispatch":
        x = s["x"].double() if s["index"] is None else s["x"].double()[s["index"].long()]
        got = [_exact_rows(x, case["fmt"])] if case["want"] != "transposed" else []
        return got + ([_exact_columns(x, s["sizes"], case["fmt"])] if case["want"] != "rows" else [])
    if op == "grouped":
        got, at = torch.empty((case["rows"], case["N"]), dtype=torch.float64, device=DEV), 0
        for e, n in enumerate(s["sizes"]):
            if n:
                a = _exact_operand(s["a"][at:at + n], s["sa"][:, at:at + n], case["a_fmt"])
                b = _exact_operand(s["b"][e], s["sb"][e], case["b_fmt"], case["b_block_rows"])
                got[at:at + n] = case["alpha"] * (a @ b.t().contiguous())
            at += n
        return got if d is None else got + d.double()
    got, at, word = torch.zeros((case["groups"], case["m"], case["n"]), dtype=torch.float64, device=DEV), 0, 0
    for e, n in enumerate(s["sizes"]):
        if n:
            end, last = at + _up(n, 128), word + _up(n, 512) // 512
            a = _exact_operand(s["a"][:, at:end], s["sa"][word:last], case["a_fmt"])
            b = _exact_operand(s["b"][:, at:end], s["sb"][word:last], case["b_fmt"])
            got[e] = a @ b.t().contiguous()
            at, word = end, last
    return got if d is None else got + d.double()
