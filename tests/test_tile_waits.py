"""Where the tiled block-of-128 kernel waits for its fragment reads (CPU, from its source).

The reads of fragments and scale words from LDS are inline assembly: the compiler takes their registers
as written when a read is issued, and may copy them in any code of its own.  So none may be in flight where the
kernel looks up a tile, which is the compiler's code (searches, divisions, table loads).
"""
import os
import re

SRC = os.path.join(os.path.dirname(__file__), "..", "block_scaled_precision_fp8_amd", "csrc", "gemm_block128_tile.h")


def source():
    return re.sub(r"//[^\n]*", "", open(SRC).read())


def test_the_loader_waits_before_it_looks_for_its_next_tile():
    body = re.search(r"auto advance = \[&\]\(\) \{(.*?)\n    \};", source(), re.S).group(1)
    at = body.index("lds_wait();")
    assert at < body.index("next_tile(") and at < body.index("locate(")
    # (of every kind of product, on every tile that it leaves)
    assert "constexpr" not in body[:at] and body[:at].count("if (") == 1


def test_the_first_fragments_have_arrived_before_the_next_tile_is_looked_up():
    text = source()
    start, end = text.index("bool stores = false;"), text.index("there = locate(next)")
    first = text.index("read_one(R, fr[0], C0, C0)")
    assert first < start < end
    # 16-bit outputs: nothing is read after the wait; FP32 output: the wait ends the reads of half 1
    sixteen, wide = text[first:start].split("} else {")[:2]
    assert "lds_wait();" in sixteen
    assert wide.index("lds_wait();") > wide.rindex("read_half(")
    # and between tiles: the loop's last reads are waited for before the epilogue
    loop = text[end:text.index("Epilogue fin = ep;")]
    assert loop.rindex("lds_wait();") > loop.rindex("run_stage(")
