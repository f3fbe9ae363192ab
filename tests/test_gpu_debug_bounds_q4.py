"""4-bit products through the debug-bounds build (libexl3_debug.so): their
kernels check every access to the packed words, scales, zero points, inputs,
workspace and results; in-range cases match the definition and find nothing."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


def test_4_bit_products_in_the_debug_bounds_build():
    lib = os.path.join(ROOT, "gemm_exl3_gemv_b200", "libexl3_debug.so")
    assert os.path.exists(lib), "build the library first (python -m gemm_exl3_gemv_b200.build)"
    out = subprocess.run([sys.executable, os.path.join(HERE, "debug_bounds_q4_cases.py")], cwd=ROOT,
                         env=dict(os.environ, EXL3_LIBRARY=lib), capture_output=True, text=True, timeout=600)
    assert out.returncode == 0, out.stdout[-2000:] + out.stderr[-3000:]
    assert "debug-bounds 4-bit cases ok" in out.stdout
