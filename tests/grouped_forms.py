"""The rule by which the grouped products choose their kernel form, with the costs read from its source
(csrc/gemm_grouped.hip), so that a test can say which form a call reaches."""
import os
import re

SRC = os.path.join(os.path.dirname(__file__), "..", "block_scaled_precision_fp8_amd", "csrc", "gemm_grouped.hip")


def costs():
    """Per tiled form of products by row: (name, rows, columns, stage, stage of FP32 output, tile)."""
    text = open(SRC).read()
    body = re.search(r"kCost\[3\] = \{(.*?)\};", text, re.S).group(1)
    rows = re.findall(r"\{(\w+), (\d+), (\d+), ([\d.e]+), ([\d.e]+), ([\d.]+)\}", body)
    assert len(rows) == 3
    return [(n, int(a), int(b), *map(float, c)) for n, a, b, *c in rows]


def rows_form(M, N, K, groups, wide, fast):
    used, stages = min(M, groups), max(1.0, K / 128)
    weights = used * N * K / 5.0e6

    def tiles(r):
        return max(used, M / r + used / 2)

    best, form = 4 + max(used * N * K / 6.0e6, tiles(16) * (N / 16) * K * 32 / 10.0e6), "FEW"
    for name, r, c, stage, stage_f32, tile in costs():
        if name == "T256" and (wide or not fast):
            continue
        n = tiles(r) * max(1.0, N / c) / 256
        n = float(int(n + 1)) if name == "T256" else max(1.0, n)
        p = n * (stages * (stage_f32 if wide else stage) + tile)
        t = 4 + max(weights, p) + 0.3 * min(weights, p)
        if t < best:
            best, form = t, name
    return form


def columns_form(M, N, columns, groups, wide, fast):
    text = open(SRC).read()
    assert "few <= 768 ? 0.22 * blocks + 1.5 : few / 768 * (0.22 * blocks + 3.7)" in text
    assert "(wide ? 0.88 : 0.56) + 2.5" in text and "(wide ? 3.05 : 1.35) + 9.0" in text
    blocks = max(1.0, columns / 128 / groups)

    def tiles(s):
        return (M + s - 1) // s * ((N + s - 1) // s) * groups

    few = tiles(32)
    best, form = 4 + (0.22 * blocks + 1.5 if few <= 768 else few / 768 * (0.22 * blocks + 3.7)), "FEW"
    t = 4 + max(1.0, tiles(128) / 256) * (blocks * (0.88 if wide else 0.56) + 2.5)
    if t < best:
        best, form = t, "T128"
    t = 4 + (tiles(256) + 255) // 256 * (blocks * (3.05 if wide else 1.35) + 9.0)
    return "T256" if fast and t < best else form
