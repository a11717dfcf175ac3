"""Build libbsfp8.so (the HIP kernels and their C ABI) for gfx950, in-tree.

Every HIP source is compiled with packed-FP32 instruction generation disabled
(``-packed-fp32-ops``) and linked into one shared library next to this file."""
import os
import subprocess
import sys
import tempfile
import time

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libbsfp8.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"
# (the longest first: they are compiled eight at a time)
SOURCES = ["gemm_grouped_wgrad_4x4_f32.hip", "gemm_block128_4x4.hip", "gemm_grouped_2x2.hip", "gemm_grouped_wgrad_2x2.hip",
           "gemm_grouped_4x4.hip", "gemm_grouped_wgrad_4x4.hip", "gemm_grouped_1x2.hip", "gemm_fp8_big.hip",
           "api.hip", "quantize.hip", "gemm_fp8.hip", "gemm_fp8_outer.hip", "gemm_mxfp4.hip", "gemm_mx.hip",
           "quantize_block128.hip", "gemm_block128.hip", "gemm_block128_rows.hip", "gemm_block128_4x2.hip",
           "gemm_block128_3x2.hip", "gemm_block128_2x2.hip", "adamw.hip", "rmsnorm.hip", "quantize_grouped.hip",
           "gemm_grouped.hip", "gemm_grouped_rows.hip", "gemm_grouped_wgrad.hip"]


def build(verbose: bool = False, jobs: int = 8) -> str:
    flags = ["--offload-arch=" + ARCH, "-O3", "-std=c++17", "-fPIC", "-Wall",
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
             "-I", os.path.join(HERE, "..", "include")]
    objs = []
    procs = []
    for src in SOURCES:
        obj = os.path.join(CSRC, src.replace(".hip", ".o"))
        cmd = [HIPCC, *flags, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        # a file, not a pipe: nobody reads it before the compiler ends
        out = tempfile.TemporaryFile()
        p = subprocess.Popen(cmd, stdout=out, stderr=subprocess.STDOUT)
        p.stdout = out
        procs.append((src, p))
        objs.append(obj)
        while len(procs) >= jobs:
            _reap(procs, verbose)
    while procs:
        _reap(procs, verbose)
    link = [HIPCC, "--offload-arch=" + ARCH, "-shared", "-fPIC", "-o", LIB + ".tmp", *objs]
    if verbose:
        print(" ".join(link), flush=True)
    subprocess.run(link, check=True)
    os.replace(LIB + ".tmp", LIB)
    return LIB


def _reap(procs, verbose):
    """Takes the compilers that have ended off the list, after waiting for one."""
    while all(p.poll() is None for _, p in procs):
        time.sleep(0.05)
    for src, p in [q for q in procs if q[1].returncode is not None]:
        procs.remove((src, p))
        p.stdout.seek(0)
        text = p.stdout.read().decode(errors="replace")
        # the host pass does not know the device-only feature flag; that note is harmless
        lines = [l for l in text.splitlines() if "not a recognized feature" not in l]
        if p.returncode != 0:
            for _, q in procs:
                q.kill()
            raise RuntimeError(f"hipcc failed for {src}:\n" + "\n".join(lines))
        if verbose and lines:
            print("\n".join(lines))


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
