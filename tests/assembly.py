"""Checks of the built library's gfx950 code, over the control flow of each kernel, for what the hardware leaves to
software: how soon a matrix instruction's result may be used, and that a read from LDS has arrived.

The compiler sees to both for its own instructions, but not where inline assembly is a side; and it has been seen
to leave the first out behind a loop that may be skipped.
"""
import glob
import os
import re
import subprocess

OBJDUMP = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin", "llvm-objdump")

#: Wait states between a matrix instruction and the first use of its result, by the passes of the matrix core that it
#: takes: 5 for two passes (16 x 16 x 32), 12 for eight, 20 for sixteen (FP8 operands of 32 x 32 x 64; FP4 ones take eight).
NEED = {"v_mfma_f32_16x16x32_bf16": 5, "v_mfma_scale_f32_16x16x128_f8f6f4": 12, "v_mfma_f32_32x32x16_bf16": 12}
NEED.update({f"v_mfma_f32_32x32x16_{a}_{b}": 12 for a in ("fp8", "bf8") for b in ("fp8", "bf8")})
NEED_FP8, NEED_FP4 = 20, 12

_REG = re.compile(r"\b([va])(?:\[(\d+):(\d+)\]|(\d+)\b)")
_VECTOR = ("v_", "ds_", "global_", "buffer_", "flat_", "scratch_")


def registers(text):
    out = []
    for kind, a, b, one in _REG.findall(text):
        out += [kind + one] if one else [f"{kind}{i}" for i in range(int(a), int(b) + 1)]
    return out


def need(instruction):
    op = instruction.split()[0]
    if op in NEED:
        return NEED[op]
    assert op.endswith("32x32x64_f8f6f4"), f"no entry for {op}"
    return NEED_FP4 if "cbsz:4 blgp:4" in instruction else NEED_FP8


def disassemble(library, folder):
    """The text of each of the library's code objects (extracted in `folder`)."""
    os.symlink(os.path.abspath(library), os.path.join(folder, "library.so"))
    subprocess.run([OBJDUMP, "--offloading", "library.so"], cwd=folder, check=True, stdout=subprocess.DEVNULL)
    for f in sorted(glob.glob(os.path.join(folder, "library.so.*gfx950"))):
        yield subprocess.run([OBJDUMP, "-d", f], check=True, capture_output=True, text=True).stdout


def kernels(text):
    """(name, [(offset, instruction, the offset that it branches to or None)]) of each function."""
    for m in re.finditer(r"^([0-9a-f]+) <(\w+)>:\n(.*?)(?=^[0-9a-f]+ <|\Z)", text, re.S | re.M):
        start, name, code = int(m.group(1), 16), m.group(2), []
        for line in m.group(3).split("\n"):
            ins, _, note = line.partition("//")
            ins = ins.strip()
            if not note or not ins:
                continue
            to = re.search(r"<" + name + r"(?:\+0x([0-9a-f]+))?>", note) if re.match(r"s_c?branch", ins) else None
            code.append((int(note.split(":")[0], 16) - start, ins, int(to.group(1) or "0", 16) if to else None))
        yield name, code


def blocks(code):
    """[instructions], [numbers of the blocks that follow]."""
    heads = {to for _, _, to in code if to is not None}
    out, at = [[]], {}
    for offset, ins, to in code:
        if offset in heads and out[-1]:
            out.append([])
        if not out[-1]:
            at[offset] = len(out) - 1
        out[-1].append((ins, to))
        if re.match(r"s_(cbranch|branch|endpgm|setpc)", ins):
            out.append([])
    follow = []
    for i, b in enumerate(out):
        ins, to = b[-1] if b else ("", None)
        next_ones = [at[to]] if to is not None else []
        if not re.match(r"s_(branch|endpgm|setpc)", ins) and i + 1 < len(out):
            next_ones.append(i + 1)
        follow.append(next_ones)
    return [[ins for ins, _ in b] for b in out], follow


def _flow(code, step, worse):
    """Runs step(state, block) -> state over the blocks until nothing changes; `worse(a, b)`: a is to be kept."""
    bodies, follow = blocks(code)
    entry, work = {0: {}}, [0]
    while work:
        i = work.pop()
        out = step(entry[i], bodies[i])
        for j in follow[i]:
            if j not in entry:
                entry[j] = dict(out)
                work.append(j)
                continue
            new = {r: v for r, v in out.items() if r not in entry[j] or worse(v, entry[j][r])}
            if new:
                entry[j].update(new)
                work.append(j)


def early_uses(code):
    """(wait states, needed, matrix instruction, its reader) of the results that are used too soon."""
    found = {}

    def step(entry, body):
        # register -> (the time of its matrix instruction, that instruction); the block starts at 0
        live, now = {r: (-age, m) for r, (age, m) in entry.items()}, 0
        for ins in body:
            op, _, rest = ins.partition(" ")
            parts = re.split(r",(?![^\[]*\])", rest)
            used, written = [], []
            if op.startswith("v_mfma"):
                # (an accumulator passes from one matrix instruction to the next by itself)
                used, written = registers(",".join(parts[1:3] + parts[4:])), registers(parts[0])
            elif op.startswith(_VECTOR):
                used, written = registers(rest), registers(parts[0]) if op.startswith("v_") else []
            for r in used:
                if r in live and now - live[r][0] < need(live[r][1]):
                    t, m = live[r]
                    found[(m, ins)] = min((now - t, need(m), m, ins), found.get((m, ins), (99,)))
            for r in written:
                live.pop(r, None)
            now += int(rest, 0) + 1 if op == "s_nop" else 1
            if op.startswith("v_mfma"):
                for r in written:
                    live[r] = (now, ins)
        return {r: (now - t, m) for r, (t, m) in live.items() if now - t < 24}

    _flow(code, step, lambda a, b: need(a[1]) - a[0] > need(b[1]) - b[0])
    return sorted(found.values())

def unfinished_reads(code):
    """(the read, the instruction that uses its registers) where nothing waited for a read from LDS."""
    found = set()

    def step(entry, body):
        # register -> (how many LDS operations were issued after its read, the read)
        live = dict(entry)
        for ins in body:
            op, _, rest = ins.partition(" ")
            if op == "s_waitcnt":
                m = re.search(r"lgkmcnt\((\d+)\)", rest)
                if m:
                    live = {r: v for r, v in live.items() if v[0] < int(m.group(1))}
                continue
            if op.startswith(_VECTOR):
                for r in registers(rest):
                    if r in live:
                        found.add((live[r][1], ins))
                        del live[r]
            if op.startswith(("ds_", "s_load", "s_buffer_load", "flat_")):
                live = {r: (n + 1, read) for r, (n, read) in live.items()}
            if op.startswith(("ds_read", "ds_bpermute", "ds_permute", "ds_swizzle")):
                for r in registers(rest.split(",")[0] if "[" not in rest.split(",")[0] else rest[:rest.index("]") + 1]):
                    live[r] = (0, ins)
        return live

    _flow(code, step, lambda a, b: a[0] < b[0])
    return sorted(found)
