"""Refusals of the block-of-128 and AdamW entry points, from the host's checks (CPU): every call
here returns before anything could be launched."""
import ctypes

import pytest

import block_scaled_precision_fp8_amd as bs

OK, INVALID, UNSUPPORTED = 0, 1, 2
E4M3, E5M2, MXFP4 = 0, 1, 2
F32, BF16, F16 = 0, 1, 2
P = 0x10000


@pytest.fixture(scope="module")
def L():
    return bs.lib()


def test_quantize(L):
    names = "x x_type rows k ld block_rows fmt codes scales codes_t scales_t stream".split()
    good = dict(x=P, x_type=BF16, rows=0, k=64, ld=64, block_rows=1, fmt=E4M3, codes=P, scales=P, codes_t=0,
                scales_t=0, stream=None)

    def call(**kw):
        return L.fp8_quantize_block128(*[{**good, **kw}[n] for n in names])

    assert call() == OK                                     # no rows: nothing to do
    assert call(rows=4, k=0, ld=0) == OK
    assert call(fmt=MXFP4) == UNSUPPORTED and call(fmt=9) == UNSUPPORTED
    assert call(x_type=3) == UNSUPPORTED
    for b in (0, 2, 64, 127, 256, -1):
        assert call(block_rows=b) == UNSUPPORTED
    r = dict(rows=4)
    assert call(rows=-1) == INVALID and call(**r, k=-1) == INVALID
    assert call(**r, ld=63) == INVALID
    assert call(rows=1 << 31) == INVALID and call(**r, k=1 << 31, ld=1 << 31) == INVALID
    assert call(**r, x=0) == INVALID
    assert call(**r, x=P + 1) == INVALID and call(**r, x=P + 2, x_type=F32) == INVALID
    assert call(rows=(1 << 31) - 1, k=1, ld=1) == INVALID   # 2^24 workgroups of 256: one too many for a launch
    assert call(**r, codes=0, scales=0) == INVALID          # no orientation
    assert call(**r, codes=0) == INVALID and call(**r, scales=0) == INVALID
    assert call(**r, codes_t=P) == INVALID and call(**r, scales_t=P) == INVALID
    assert call(**r, codes=P + 8) == INVALID and call(**r, scales=P + 2) == INVALID
    assert call(**r, codes_t=P + 8, scales_t=P) == INVALID


def test_gemm(L):
    names = ("M N K a_fmt a a_scales a_block_rows b_fmt b b_scales b_block_rows alpha c ldc beta out d ldd "
             "stream").split()
    good = dict(M=0, N=8, K=64, a_fmt=E4M3, a=P, a_scales=P, a_block_rows=1, b_fmt=E5M2, b=P, b_scales=P,
                b_block_rows=128, alpha=1.0, c=0, ldc=0, beta=0.0, out=BF16, d=P, ldd=8, stream=None)

    def call(**kw):
        return L.scaled_gemm_block128(*[{**good, **kw}[n] for n in names])

    assert call() == OK and call(M=8, N=0) == OK
    assert call(a_fmt=MXFP4) == UNSUPPORTED and call(b_fmt=-1) == UNSUPPORTED and call(out=3) == UNSUPPORTED
    assert call(a_block_rows=32) == UNSUPPORTED and call(b_block_rows=0) == UNSUPPORTED
    m = dict(M=8)
    assert call(M=-1) == INVALID and call(N=-1) == INVALID and call(K=-32) == INVALID
    assert call(**m, K=48) == INVALID
    assert call(**m, K=1 << 23) == UNSUPPORTED
    assert call(M=1 << 31) == INVALID
    assert call(M=(1 << 31) - 256) == INVALID and call(M=8, N=(1 << 31) - 256, ldd=1 << 31) == INVALID
    assert call(M=(1 << 31) - 512, N=(1 << 31) - 512, ldd=1 << 31) == INVALID  # more tiles than 32 bits count
    assert call(**m, ldd=7) == INVALID and call(**m, d=0) == INVALID and call(**m, d=P + 1) == INVALID
    assert call(**m, d=P + 2, out=F32) == INVALID
    assert call(**m, beta=1.0) == INVALID                   # beta without C
    assert call(**m, beta=1.0, c=P, ldc=7) == INVALID and call(**m, beta=1.0, c=P + 1, ldc=8) == INVALID
    for k in ("a", "b", "a_scales", "b_scales"):
        assert call(**m, **{k: 0}) == INVALID
        assert call(**m, **{k: P + 2}) == INVALID


class Tensor(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("p", "g", "m", "v", "ms", "vs")] + [("n", ctypes.c_int64)]


def test_adamw(L):
    def tensors(*kw):
        base = dict(p=P, g=P + 0x10000, m=P + 0x20000, v=P + 0x30000, ms=0, vs=0, n=0)
        return (Tensor * len(kw))(*[Tensor(**{**base, **k}) for k in kw])

    def call(t=None, count=None, p=F32, g=BF16, state=0, args=True, **kw):
        t = tensors({}) if t is None else t
        a = bs._AdamWArgs(**{**dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1, step=1), **kw})
        return L.adamw_step(ctypes.addressof(t), len(t) if count is None else count, p, g, state,
                            ctypes.addressof(a) if args else None, None)

    assert call() == OK and call(count=0) == OK             # empty tensors: nothing to do
    assert L.adamw_step(None, 1, F32, F32, 0, ctypes.addressof(bs._AdamWArgs(step=1)), None) == INVALID
    assert call(args=False) == INVALID and call(count=-1) == INVALID
    assert call(p=F16) == UNSUPPORTED and call(p=7) == UNSUPPORTED and call(g=7) == UNSUPPORTED
    assert call(state=2) == UNSUPPORTED
    for k, bad in (("beta1", (1.0, -0.1, float("nan"))), ("beta2", (1.0, -0.1, float("nan"))),
                   ("eps", (-1.0, float("nan"), float("inf"))), ("lr", (float("nan"), float("inf"))),
                   ("weight_decay", (float("nan"),)), ("step", (0, -3)), ("lr_dev", (P + 2,)),
                   ("step_dev", (P + 4,)), ("grad_scale", (P + 1,)), ("found_inf", (P + 3,))):
        for b in bad:
            assert call(**{k: b}) == INVALID, (k, b)
    n = dict(n=100)
    for k in ("p", "g", "m", "v"):
        assert call(tensors({**n, k: 0})) == INVALID
        assert call(tensors({**n, k: P + 0x40001})) == INVALID
    assert call(tensors(dict(n=-1))) == INVALID and call(tensors(dict(n=1 << 41))) == INVALID
    assert call(tensors(n), state=1) == INVALID             # FP8 states without scales
    # overlaps: two tensors' parameters, a state with a gradient, a tensor given twice, scales inside codes
    far = dict(p=P + 0x100000, g=P + 0x110000, m=P + 0x120000, v=P + 0x130000, n=100)
    assert call(tensors(n, {**far, "p": P + 396})) == INVALID
    assert call(tensors(n, {**far, "m": P + 0x10000})) == INVALID
    assert call(tensors(n, n)) == INVALID
    assert call(tensors({**n, "ms": P + 0x20010, "vs": P + 0x50000}), state=1) == INVALID
    assert call(tensors({**n, "p": P + 0x20000})) == INVALID
    # device scalars inside what the step writes
    for k, at in (("lr_dev", P + 396), ("step_dev", P + 0x20000), ("grad_scale", P + 0x30000 + 8), ("found_inf", P)):
        assert call(tensors(n), **{k: at}) == INVALID, k


def test_binding_refusals():
    import torch
    x = torch.zeros((4, 64))
    q, s = torch.zeros((4, 64), dtype=torch.uint8), torch.zeros((1, 4, 4), dtype=torch.uint8)
    for call in (lambda: bs.fp8_quantize_block128(x), lambda: bs.scaled_gemm_block128(q, s, q, s),
                 lambda: bs.adamw_step([x], [x], [x], [x]), lambda: bs.adamw_step([x], [x], [x], []),
                 lambda: bs.adamw_step([x], [x], [x], [x], [s], None),
                 lambda: bs.scaled_gemm_block128(q, s, q, s, "mxfp4"),
                 lambda: bs.scaled_gemm_block128(q, s, q, s, a_block_rows=2),
                 lambda: bs.adamw_states([x], "f16")):
        with pytest.raises(ValueError):
            call()
    bs.adamw_step([], [], [], [])


@pytest.mark.parametrize("state", ["f32", "fp8"])
def test_states_of_a_generator(state):
    """Parameters come as model.parameters() does: a generator, read once."""
    import torch
    params = [torch.zeros(3, 5), torch.zeros(300)]
    m, v, ms, vs = bs.adamw_states((p for p in params), state)
    assert [t.shape for t in m] == [t.shape for t in v] == [p.shape for p in params]
    assert (ms is None and vs is None) if state == "f32" else [t.numel() for t in ms] == [t.numel() for t in vs] == [1, 3]


def test_adamw_without_host_memory():
    """The overlap check of many tensors sorts their ranges in host memory; without it the call says
    so instead of blaming its arguments.  (The last two tensors share their parameters, so that the
    call is refused either way; in a process of its own, whose address space is limited for the call.)"""
    import subprocess
    import sys
    code = """
import ctypes, resource, struct, sys
import block_scaled_precision_fp8_amd as bs
L = bs.lib()
def status(count, leave):
    at = 1 << 40
    rows = [struct.pack("<7q", at + 64 * i, at + 64 * i + 16, at + 64 * i + 32, at + 64 * i + 48, 0, 0, 1) for i in range(count)]
    rows[-1] = rows[-2]
    t = ctypes.create_string_buffer(b"".join(rows))
    del rows
    a = bs._AdamWArgs(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, step=1)
    old = resource.getrlimit(resource.RLIMIT_AS)
    if leave:
        pages = int(open("/proc/self/statm").read().split()[0])
        resource.setrlimit(resource.RLIMIT_AS, (pages * 4096 + leave, old[1]))
    got = L.adamw_step(ctypes.addressof(t), count, 0, 0, 0, ctypes.addressof(a), None)
    resource.setrlimit(resource.RLIMIT_AS, old)
    return got
for case in ((20, 0), (90, 0), (97, 0), (98, 0), (2000, 0), (1 << 20, 0), (1 << 20, 1 << 20)):
    print(status(*case), end=" ")
"""
    root = bs.__file__.rsplit("/", 2)[0]
    out = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=100)
    assert out.stdout.split() == ["1"] * 6 + ["4"], out.stdout + out.stderr
    assert bs.lib().bsfp8_status_string(4) == b"BSFP8_ERR_NO_MEMORY"
