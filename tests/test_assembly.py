"""The built library's gfx950 code, kernel by kernel (CPU): see assembly.py for what is checked, and why."""
import concurrent.futures

import pytest

import block_scaled_precision_fp8_amd as bs
from assembly import disassemble, early_uses, kernels, unfinished_reads


def _check(text):
    """Per kernel with matrix instructions: its name, the uses of results that come too soon and of LDS reads not waited for."""
    return [(name, early_uses(code), unfinished_reads(code)) for name, code in kernels(text) if any("v_mfma" in ins for _, ins, _ in code)]


@pytest.fixture(scope="module")
def checked(tmp_path_factory):
    objects = list(disassemble(bs.LIB_PATH, str(tmp_path_factory.mktemp("objects"))))
    with concurrent.futures.ProcessPoolExecutor(4) as pool:
        return [k for part in pool.map(_check, objects) for k in part]


def test_results_are_not_used_too_soon(checked):
    assert len(checked) > 300
    for name, early, _ in checked:
        assert not early, f"{name}: {len(early)} uses, the first after {early[0][0]} of {early[0][1]} wait states: {early[0][2]} | {early[0][3]}"


def test_reads_from_lds_have_arrived(checked):
    for name, _, reads in checked:
        assert not reads, f"{name}: {len(reads)} uses of reads in flight: {reads[0][0]} | {reads[0][1]}"


def code_of(text):
    """Code as kernels() gives it, of lines of instructions with labels ("1:") and branches to them ("1f")."""
    lines, at = text.strip().split("\n"), {}
    n = 0
    for line in lines:
        if line.endswith(":"):
            at[line[:-1]] = 4 * n
        else:
            n += 1
    out = []
    for line in lines:
        if not line.endswith(":"):
            to = at[line.split()[1]] if line.startswith(("s_cbranch", "s_branch")) else None
            out.append((4 * len(out), line, to))
    return out


LOOP = """head:
v_mfma_scale_f32_16x16x128_f8f6f4 v[2:5], v[28:35], v[36:43], v[2:5], v18, v13 op_sel_hi:[0,0,0]
s_cbranch_scc0 head
s_branch out
skipped:
v_mov_b32_e32 v9, v1
out:
{wait}
ds_write_b128 v22, v[2:5]
s_cbranch_vccnz skipped
s_endpgm"""


@pytest.mark.parametrize("wait,states", [("s_nop 8", 11), ("s_nop 0", 3), ("s_mov_b32 s0, 0", 3), ("s_nop 9", None), ("s_nop 15", None)])
def test_the_count_follows_the_control_flow(wait, states):
    """The result reaches its reader around a block that is jumped over: two branches and the wait."""
    assert [e[0] for e in early_uses(code_of(LOOP.format(wait=wait)))] == ([] if states is None else [states])


def test_the_count_knows_the_instructions():
    def uses(m, n, reader):
        return [(e[0], e[1]) for e in early_uses(code_of(f"{m}\ns_nop {n - 1}\n{reader}\ns_endpgm"))]
    fp8 = "v_mfma_f32_32x32x64_f8f6f4 a[0:15], v[0:7], v[8:15], a[0:15] blgp:1"
    fp4 = "v_mfma_scale_f32_32x32x64_f8f6f4 a[0:15], v[0:3], v[8:11], a[0:15], v20, v21 op_sel_hi:[0,0,0] cbsz:4 blgp:4"
    read = "v_accvgpr_read_b32 v40, a3"
    assert uses(fp8, 16, read) == [(16, 20)] and uses(fp4, 11, read) == [(11, 12)] and not uses(fp4, 12, read)
    # another register, a result overwritten in between, and the next product's accumulator are no uses
    assert not uses(fp8, 2, "v_accvgpr_read_b32 v40, a16") and not uses(fp8, 2, fp8)
    assert uses(fp8, 2, "v_mfma_f32_32x32x16_bf16 a[16:31], a[0:3], v[8:11], a[16:31]") == [(2, 20)]


@pytest.mark.parametrize("wait,reads", [("lgkmcnt(0)", 0), ("lgkmcnt(1)", 0), ("lgkmcnt(2)", 1), ("vmcnt(0)", 1), ("vmcnt(3) lgkmcnt(0)", 0)])
def test_the_reads_are_counted_in_order(wait, reads):
    """Of three LDS operations the second is waited for, or not, and used around a loop."""
    text = f"""ds_read_b32 v1, v0
head:
ds_read_b128 v[4:7], v0 offset:16
ds_write_b32 v0, v9
s_waitcnt {wait}
v_add_u32_e32 v10, v10, v6
s_cbranch_scc0 head
s_endpgm"""
    assert len({r for r, _ in unfinished_reads(code_of(text))}) == reads


def test_a_register_written_over_a_read_in_flight_counts():
    assert unfinished_reads(code_of("ds_read_b64 v[4:5], v0\nv_mov_b32_e32 v5, 0\ns_endpgm"))
    assert not unfinished_reads(code_of("ds_read_b64 v[4:5], v0\nv_mov_b32_e32 v6, 0\ns_waitcnt lgkmcnt(0)\nv_mov_b32_e32 v5, v4\ns_endpgm"))
