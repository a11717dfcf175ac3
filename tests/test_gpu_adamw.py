"""Parity of adamw_step with its references (MI355X).

Bit for bit with the float32 reference, whose operations are rounded one by one as the kernel's are
(the states' codes and scales included), and near the float64 one, within the sum of the roundings on
the way, each at most 2^-24 of its result."""
import numpy as np
import pytest

import block_scaled_precision_fp8_amd as bs
from gpu_common import from_dev, say
from oracle import block128 as ref

pytestmark = pytest.mark.gpu
HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1)


def make(sizes, state, p_type, g_type, seed):
    import torch
    g = np.random.default_rng(seed)
    t = dict(p=[], g=[], m=[], v=[], ms=[], vs=[])
    for n in sizes:
        t["p"].append(torch.from_numpy(g.standard_normal(n).astype(np.float32) * 0.02).to(p_type).cuda())
        gr = g.standard_normal(n) * 10.0 ** g.uniform(-5, -1, n)
        gr[g.random(n) < 0.1] = 0
        t["g"].append(torch.from_numpy(gr.astype(np.float32)).to(g_type).cuda())
        m, r = g.standard_normal(n).astype(np.float32) * 1e-3, np.abs(g.standard_normal(n)).astype(np.float32) * 1e-2
        if state == "f32":
            t["m"].append(torch.from_numpy(m).cuda())
            t["v"].append(torch.from_numpy(r * r).cuda())
        else:
            for x, k in ((m, "m"), (r, "v")):
                c, s = ref.round_state(x, np.zeros(n, np.uint64), False)
                t[k].append(torch.from_numpy(c).cuda())
                t[k + "s"].append(torch.from_numpy(s).cuda())
    return t


def expected(t, i, state, seed, step, gs, dtype):
    """(p', m', v' or codes and scales) of tensor i; p' as float32 or, for bf16, its rounded value."""
    import torch
    p, g = (t[k][i].float().cpu().numpy() for k in ("p", "g"))
    n = p.size
    if state == "f32":
        m, v = from_dev(t["m"][i]), from_dev(t["v"][i])
    else:
        m = ref.state_values(from_dev(t["m"][i]), from_dev(t["ms"][i]))
        r = ref.state_values(from_dev(t["v"][i]), from_dev(t["vs"][i])).astype(dtype)
        v = r * r
    p, m, v, r = ref.adamw(p, g, m, v, HP, step, gs, dtype)
    bits = ref.noise(n, seed, step, i)
    if t["p"][i].dtype == torch.bfloat16 and dtype == np.float32:
        p = ref.round_bf16(p, bits & np.uint64(0xFFFF))
    if state == "f32":
        return p, m, v
    return (p,) + ref.round_state(m, bits & np.uint64(0xFFFF), False) + ref.round_state(r, bits >> np.uint64(16), True)


SIZES = [1, 5, 127, 128, 129, 2047, 2048, 2049, 5000]


@pytest.mark.parametrize("state", ["f32", "fp8"])
@pytest.mark.parametrize("p_type", ["float32", "bfloat16"])
@pytest.mark.parametrize("g_type", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("step", [1, 1000])
def test_step(state, p_type, g_type, step):
    import torch
    t = make(SIZES, state, getattr(torch, p_type), getattr(torch, g_type), 1)
    gs = torch.tensor([0.75], device="cuda")
    fp8 = state == "fp8"
    want = [expected(t, i, state, 11, step, 0.75, np.float32) for i in range(len(SIZES))]
    wide = [expected(t, i, state, 11, step, 0.75, np.float64) for i in range(len(SIZES))]
    update = []
    for i, n in enumerate(SIZES):
        g = np.abs(t["g"][i].double().cpu().numpy() * 0.75)
        if fp8:
            m = ref.state_values(from_dev(t["m"][i]), from_dev(t["ms"][i]))
            v = ref.state_values(from_dev(t["v"][i]), from_dev(t["vs"][i])) ** 2
        else:
            m, v = from_dev(t["m"][i]).astype(np.float64), from_dev(t["v"][i]).astype(np.float64)
        b1, c1, b2, c2, _, size, rbc, eps = ref.constants(**HP, step=step)
        update.append(size * (b1 * np.abs(m) + c1 * g) / (np.sqrt(b2 * v + c2 * g * g) * rbc + eps))
    say(f"adamw_step {state} {p_type} {g_type} step {step}")
    bs.adamw_step(t["p"], t["g"], t["m"], t["v"], t["ms"] if fp8 else None, t["vs"] if fp8 else None, step=step,
                  grad_scale=gs, seed=11, **HP)
    for i, n in enumerate(SIZES):
        got = [t["p"][i].float()] + ([t["m"][i], t["ms"][i], t["v"][i], t["vs"][i]] if fp8 else [t["m"][i], t["v"][i]])
        for j, (a, b) in enumerate(zip(got, want[i])):
            assert np.array_equal(from_dev(a), b), f"size {n}, output {j}"
        # p (1 - lr wd): the factor and the product; the difference: p'.  The update's numerator: b1, c1,
        # g, both products, their sum, size and its product (8 of size (b1 |m| + c1 |g|)); its denominator:
        # b2, c2, two products and a square, halved by the root, the root, rbc and its product, eps, the sum
        # (8); the quotient (1); and once more for what these leave out (products of roundings)
        p64, got_p = wide[i][0], from_dev(got[0])
        bound = 2.0 ** -24 * (3 * np.abs(p64) + 3 * update[i] + 18 * update[i])
        if p_type == "bfloat16":
            bound += 2.0 ** -7 * np.abs(p64)       # the cut bits carry or not: under one step
        assert np.all(np.abs(got_p - p64) <= bound)


def test_many_tensors_unaligned_views_and_guards():
    """More tensors than a launch takes, empty ones, views at odd addresses, nothing outside touched."""
    import torch
    g = np.random.default_rng(0)
    sizes = [int(n) for n in g.integers(0, 400, 130)]
    for state in ("f32", "fp8"):
        t = make(sizes, state, torch.float32, torch.bfloat16, 2)
        fp8 = state == "fp8"
        # move every tensor into one buffer per kind, one element apart
        flat = {}
        for k in ("p", "g", "m", "v") + (("ms", "vs") if fp8 else ()):
            src = t[k]
            buf = torch.full((sum(x.numel() + 3 for x in src) + 3,), 7, dtype=src[0].dtype, device="cuda")
            at, views = 3, []
            for x in src:
                buf[at:at + x.numel()] = x
                views.append(buf[at:at + x.numel()])
                at += x.numel() + 3
            flat[k], t[k] = buf, views
        want = [expected(t, i, state, 5, 3, 1.0, np.float32) for i in range(len(sizes))]
        say(f"adamw_step many tensors {state}")
        bs.adamw_step(t["p"], t["g"], t["m"], t["v"], t["ms"] if fp8 else None, t["vs"] if fp8 else None, step=3,
                      seed=5, **HP)
        for i, n in enumerate(sizes):
            got = [t["p"][i]] + ([t["m"][i], t["ms"][i], t["v"][i], t["vs"][i]] if fp8 else [t["m"][i], t["v"][i]])
            for a, b in zip(got, want[i]):
                assert np.array_equal(from_dev(a), b)
        for k, buf in flat.items():
            b, at = from_dev(buf), 0
            for x in t[k]:
                assert np.all(b[at:at + 3] == 7)
                at += 3 + x.numel()
            assert np.all(b[at:] == 7)


@pytest.mark.parametrize("state", ["f32", "fp8"])
def test_device_rates_found_inf_and_graph(state):
    """lr and step on the device, skipping, and a captured step that follows both."""
    import torch
    fp8 = state == "fp8"
    sizes = [300, 5000]
    t, u = (make(sizes, state, torch.float32, torch.float32, 3) for _ in range(2))
    lr, step = torch.tensor([1e-3], device="cuda"), torch.tensor([1], device="cuda")
    found = torch.zeros(1, device="cuda")
    hp = {k: v for k, v in HP.items() if k != "lr"}

    def go(x, lr, step):
        bs.adamw_step(x["p"], x["g"], x["m"], x["v"], x["ms"] if fp8 else None, x["vs"] if fp8 else None, lr=lr,
                      step=step, found_inf=found, seed=9, **hp)

    def same():
        return all(torch.equal(a, b) for k in t for a, b in zip(t[k], u[k]))

    say(f"adamw_step device rates {state}")
    # FP32 lr on both sides: the host's double is the tensor's value
    go(t, lr, step)
    go(u, lr.item(), 1)
    assert same()
    say(f"adamw_step found_inf {state}")
    found.fill_(1.0)
    go(t, lr, step)
    assert same()
    found.zero_()
    say(f"adamw_step graph {state}")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.add_(1)
        go(t, lr, step)
    assert same()
    for i in range(3):
        lr.fill_(1e-3 * (i + 1))
        for a, b in zip(t["g"], u["g"]):
            a.normal_(0, 1e-3)
            b.copy_(a)
        graph.replay()
        go(u, lr.item(), 2 + i)
        torch.cuda.synchronize()
        assert same()


def test_non_finite_gradients():
    import torch
    for state in ("f32", "fp8"):
        fp8 = state == "fp8"
        t = make([400], state, torch.float32, torch.float32, 4)
        t["g"][0][130] = float("nan")
        t["g"][0][300] = float("inf")
        say(f"adamw_step non-finite {state}")
        bs.adamw_step(t["p"], t["g"], t["m"], t["v"], t["ms"] if fp8 else None, t["vs"] if fp8 else None, step=2, **HP)
        p = from_dev(t["p"][0])
        bad = ~np.isfinite(p)
        assert bad[130] and bad.sum() <= 2 and (bad[300] or bad.sum() == 1)
        if fp8:
            assert from_dev(t["ms"][0]).tolist()[1:3] == [255, 255] and from_dev(t["vs"][0]).tolist()[1:3] == [255, 255]
            assert np.all(from_dev(t["m"][0])[128:384] == 0x7F) and not np.any(from_dev(t["m"][0])[:128] == 0x7F)


def test_second_moment_follows_the_gradients():
    """Stochastic states: after the gradients shrink tenfold, the mean of sqrt(v) falls as the FP32 one."""
    import torch
    n, steps = 1 << 14, 400
    out = {}
    for state in ("f32", "fp8"):
        g = torch.Generator(device="cuda")
        g.manual_seed(0)
        p = [torch.zeros(n, device="cuda")]
        m, v, ms, vs = bs.adamw_states(p, state)
        for i in range(steps):
            gr = [torch.randn(n, generator=g, device="cuda") * (1.0 if i < 50 else 0.1)]
            bs.adamw_step(p, gr, m, v, ms, vs, lr=1e-3, beta2=0.99, step=i + 1, seed=1)
        if state == "fp8":
            out[state] = ref.state_values(from_dev(v[0]), from_dev(vs[0]))
        else:
            out[state] = np.sqrt(from_dev(v[0]).astype(np.float64))
    # an element's r is a random walk of code steps around the true one; its mean over 2^14 elements
    # moves by well under 2%; frozen states would stay ten times too large
    a, b = out["f32"].mean(), out["fp8"].mean()
    say(f"mean sqrt(v): f32 {a:.4f} fp8 {b:.4f}")
    assert abs(b - a) <= 0.1 * a


def test_a_graph_of_the_old_parameters_is_refused():
    """Values that autograd saved before a step must not be replaced unnoticed."""
    import torch
    p = torch.ones(300, device="cuda", requires_grad=True)
    y = (p * p).sum()
    with torch.inference_mode():
        q = torch.ones(40, device="cuda")
    params = [p, q]
    say("adamw under a live graph")
    m, v, _, _ = bs.adamw_states(params)
    bs.adamw_step(params, [torch.ones_like(p.detach()), torch.ones(40, device="cuda")], m, v, lr=0.5, weight_decay=0.0)
    # 1 - 0.5 m' / sqrt(v') at step 1, eight roundings of at most 2^-24 each
    assert abs(float(p.detach()[0]) - 0.5) < 2.0 ** -21 and abs(float(q[0]) - 0.5) < 2.0 ** -21
    with pytest.raises(RuntimeError):
        y.backward()


def test_train_step_end_to_end():
    """An FP8 linear layer's step as it is used: quantise, three products, AdamW with FP8 states,
    and the new weight's codes; every stage against its reference on the stage's own inputs."""
    import torch
    T, O, I = 96, 130, 200
    g = np.random.default_rng(7)
    w = torch.from_numpy(g.standard_normal((O, I)).astype(np.float32) * 0.05).cuda()
    m, v, ms, vs = bs.adamw_states([w], "fp8")
    assert m[0].shape == w.shape and ms[0].numel() == (O * I + 127) // 128
    for step in (1, 2, 3):
        x = torch.from_numpy(g.standard_normal((T, I))).to(torch.bfloat16).cuda()
        dy = torch.from_numpy(g.standard_normal((T, O)) * 1e-3).to(torch.bfloat16).cuda()
        say(f"train step {step}")
        xq, xs, xqt, xst = bs.fp8_quantize_block128(x, "e4m3", 1, True, True)
        gqt, gst = bs.fp8_quantize_block128(dy, "e5m2", 1, False, True)
        dw = bs.scaled_gemm_block128(gqt, gst, xqt, xst, "e5m2", "e4m3", 1, 1, out="f32")
        d_ref, s_ref = ref.gemm(from_dev(gqt), from_dev(gst), "e5m2", 1, from_dev(xqt), from_dev(xst), "e4m3", 1)
        assert np.all(np.abs(from_dev(dw) - d_ref) <= (16 + T / 4) * 2.0 ** -24 * s_ref)
        t = dict(p=[w.view(-1)], g=[dw.view(-1)], m=[m[0].view(-1)], v=[v[0].view(-1)], ms=ms, vs=vs)
        want = expected(t, 0, "fp8", 3, step, 1.0, np.float32)
        bs.adamw_step([w], [dw], m, v, ms, vs, step=step, seed=3, **HP)
        for a, b in zip((w, m[0], ms[0], v[0], vs[0]), want):
            assert np.array_equal(from_dev(a).reshape(-1), b)
        wq, ws = bs.fp8_quantize_block128(w, "e4m3", 128)
        for a, b in zip((wq, ws), ref.quantize(from_dev(w), "e4m3", 128)):
            assert np.array_equal(from_dev(a), b)


def decay_cases():
    """(lr, wd) whose 64-bit product is inexact and lands on the value that makes 1 - lr wd a tie
    between two FP32 values: rounded by itself it rounds to even, contracted to an FMA it can go
    the other way.  Found by construction; lr is an FP32 value."""
    from fractions import Fraction
    g, out = np.random.default_rng(0), []
    while len(out) < 4:
        tie = (2 * int(g.integers(1 << 23, 1 << 24)) + 1) * 2.0 ** -26      # in [0.25, 0.5), between two FP32 values
        lr = float(np.float32(g.uniform(0.5, 1.0)))
        wd = (1.0 - tie) / lr
        left = 1 - Fraction(lr) * Fraction(wd) - Fraction(tie)
        if lr * wd == 1.0 - tie and left and np.float32(float(Fraction(tie) + left)) != np.float32(tie):
            out.append((lr, wd))
    return out


def test_rates_on_the_device_are_the_arguments_rates():
    """The same lr and step as device scalars and as arguments: the same bits."""
    import torch

    def pair(lr, wd, step, m0):
        got = []
        for on_device in (False, True):
            p, g = [torch.ones(300, device="cuda")], [torch.zeros(300, device="cuda")]
            m, v = [torch.full((300,), m0, device="cuda")], [torch.full((300,), 1e-6, device="cuda")]
            bs.adamw_step(p, g, m, v, lr=torch.tensor([lr], device="cuda") if on_device else lr,
                          step=torch.tensor([step], device="cuda") if on_device else step, weight_decay=wd)
            got.append(from_dev(p[0]))
        return got

    say("adamw_step decay rates at a tie")
    for lr, wd in decay_cases():
        host, dev = pair(lr, wd, 5, 0.0)
        assert np.all(host == np.float32(1.0 - lr * wd))
        assert np.array_equal(host, dev)
    for step in (1, 2, 7, 50, 999, 20011, 1 << 20):
        say(f"adamw_step rates at step {step}")
        for lr in (1e-5, 3e-4, 0.1):
            host, dev = pair(float(np.float32(lr)), 0.1, step, 1e-3)
            assert np.array_equal(host, dev)


@pytest.mark.parametrize("state", ["f32", "fp8"])
def test_shapes_that_do_not_agree_are_refused(state):
    """A gradient or state of another shape with as many elements: refused, nothing written.  Flat ones
    are taken: the same result."""
    import torch
    def fresh():
        t = make([600], state, torch.float32, torch.float32, 8)
        for k in "pgmv":
            t[k] = [t[k][0].view(20, 30)]
        return t

    def go(t):
        fp8 = state == "fp8"
        bs.adamw_step(t["p"], t["g"], t["m"], t["v"], t["ms"] if fp8 else None, t["vs"] if fp8 else None, step=2,
                      seed=4, **HP)

    t = fresh()
    say(f"adamw_step shapes {state}")
    for k, name in (("g", "grads"), ("m", "m"), ("v", "v")):
        for shape in ((30, 20), (1, 600), (20, 30, 1)):
            with pytest.raises(ValueError, match=rf"{name}\[0\] has shape"):
                go({**t, k: [t[k][0].view(shape)]})
    want = fresh()
    assert all(torch.equal(a, b) for k in t for a, b in zip(t[k], want[k]))
    go(want)
    for flat in ("g", "p", "gmv"):
        t = fresh()
        go({**t, **{k: [t[k][0].view(-1)] for k in flat}})
        assert all(torch.equal(a, b) for k in t for a, b in zip(t[k], want[k]))


@pytest.mark.parametrize("state", ["f32", "fp8"])
def test_states_count_the_step_in_their_versions(state):
    import torch
    p, g = [torch.ones(300, device="cuda")], [torch.ones(300, device="cuda")]
    states = bs.adamw_states(p, state)
    say(f"adamw_step versions {state}")
    kept = [p[0]] + [t[0] for t in states if t is not None]
    before, g0 = [t._version for t in kept], g[0]._version
    bs.adamw_step(p, g, *states)
    assert [t._version for t in kept] == [n + 1 for n in before] and g[0]._version == g0


@pytest.mark.parametrize("state", ["f32", "fp8"])
@pytest.mark.parametrize("p_type", ["float32", "bfloat16"])
def test_non_finite_values_stay_in_their_places(state, p_type):
    """NaN and infinities in gradients and parameters: NaN or infinite in the same elements of p, m and
    v (FP8 states: in the whole block of 128 of m and v), every other element as without them."""
    import torch
    fp8, dt, n = state == "fp8", getattr(torch, p_type), 700
    t, u = (make([n], state, dt, torch.float32, 4) for _ in range(2))
    inf, nan = float("inf"), float("nan")
    for i, x in ((130, nan), (300, inf), (301, -inf)):
        t["g"][0][i] = x
    for i, x in ((3, nan), (400, inf), (401, -inf)):
        t["p"][0][i] = x
    if p_type == "bfloat16":
        t["p"][0].view(torch.int16)[4] = 0x7F81         # a NaN whose set bit is the lowest
    say(f"adamw_step non-finite {state} {p_type}")
    for x in (t, u):
        bs.adamw_step(x["p"], x["g"], x["m"], x["v"], x["ms"] if fp8 else None, x["vs"] if fp8 else None, step=2,
                      seed=5, **HP)
    p, q = from_dev(t["p"][0]), from_dev(u["p"][0])
    nans = [3, 130, 300, 301] + ([4] if p_type == "bfloat16" else [])
    assert np.isnan(p[nans]).all() and p[400] == inf and p[401] == -inf
    keep = np.setdiff1d(np.arange(n), nans + [400, 401])
    assert np.array_equal(p[keep], q[keep])
    if fp8:
        for k in "mv":
            c, s = from_dev(t[k][0]), from_dev(t[k + "s"][0])
            d, e = from_dev(u[k][0]), from_dev(u[k + "s"][0])
            assert s.tolist() == [e[0], 255, 255, *e[3:]] and np.all(c[128:384] == 0x7F)
            keep = np.r_[0:128, 384:n]
            assert np.array_equal(c[keep], d[keep])
    else:
        m, v = from_dev(t["m"][0]), from_dev(t["v"][0])
        assert np.isnan(m[130]) and np.isnan(v[130]) and m[300] == inf and m[301] == -inf and np.all(v[300:302] == inf)
        keep = np.setdiff1d(np.arange(n), [130, 300, 301])
        assert np.array_equal(m[keep], from_dev(u["m"][0])[keep]) and np.array_equal(v[keep], from_dev(u["v"][0])[keep])
