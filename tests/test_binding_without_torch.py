"""The binding's C functions in a process that has no torch (CPU)."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=120)


def test_the_library_loads_without_torch():
    """lib() and the calls that take no tensor work where torch cannot be imported."""
    r = run("import sys; sys.modules['torch'] = None\n"
            "import block_scaled_precision_fp8_amd as bs\n"
            "assert bs.lib().bsfp8_version() > 0 and bs.rmsnorm_backward_workspace(4, 64) > 0\n"
            "assert bs.block128_grouped_shape(5, 7, 2) == ((7, 256), (2, 7, 4))\n"
            "assert bs.lib().fp8_quantize(None, 0, 0, 0, 0, 0, None, None, None) in (0, 1, 2)\n"
            "print('loaded')")
    assert r.returncode == 0 and r.stdout.strip() == "loaded", r.stderr


def test_torch_comes_first_where_there_is_one():
    """With torch its HIP runtime is the process's own: it is loaded before the library's."""
    r = run("import sys, block_scaled_precision_fp8_amd as bs\n"
            "assert 'torch' not in sys.modules\n"
            "bs.lib()\n"
            "assert 'torch' in sys.modules\n"
            "print('loaded')")
    assert r.returncode == 0 and r.stdout.strip() == "loaded", r.stderr
