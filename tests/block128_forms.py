"""Which form of the block-of-128 GEMM a shape takes, and how many tiles a workgroup of it computes:
the rule of csrc/gemm_block128.hip on the host, with its constants read from the source, so that the
cases of the tests keep naming the forms that they reach (test infrastructure)."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "block_scaled_precision_fp8_amd", "csrc")
NAMES = {(256, 256): "256x256", (256, 128): "256x128", (192, 128): "192x128", (128, 128): "128x128"}


def _constants():
    text = open(os.path.join(CSRC, "gemm_block128.hip")).read()
    table = text[text.index("kCost[4] = {"):text.index("const double stages")]
    cost = [tuple(float(x) for x in m) for m in re.findall(r"\{(\d+), (\d+), ([\d.e]+), ([\d.e]+), ([\d.e]+)\}", table)]
    narrow = re.search(r"BSFP8_OUT_F32 \? ([\d.e]+) : ([\d.e]+)\);", text)
    head = open(os.path.join(CSRC, "gemm_block128.h")).read()
    rows = [int(re.search(rf"kRowsMax{d} = (\d+);", head).group(1)) for d in "MN"]
    assert len(cost) == 4 and narrow
    return cost, [float(x) for x in narrow.groups()], rows


COST, NARROW, ROWS = _constants()


def up(a, b):
    return (a + b - 1) // b


def form(M, N, K, out):
    """(name, tiles of the largest workgroup)."""
    f32 = out == "f32"
    if M <= ROWS[0] and N <= ROWS[1]:
        return "rows", 1
    stages = up(K, 128)
    best, name, tiles = 4.0 + up(M, 32) * up(up(N, 32), 8) * 8 * K * 64.0 / NARROW[0 if f32 else 1], "32x32", 1
    for ra, rb, stage, stage_f32, tile in COST:
        ra, rb = int(ra), int(rb)
        n = up(M, ra) * up(N, rb)
        t = 4.0 + up(n, 256) * (stages * (stage_f32 if f32 else stage) + tile)
        if t < best:
            best, name, tiles = t, NAMES[ra, rb], 1 if (ra, rb) == (128, 128) else up(n, 256)
    return name, tiles
