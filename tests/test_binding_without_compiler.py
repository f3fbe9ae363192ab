"""The library without the compiled part of its binding (no C compiler, no
Python headers, another Python than the one it was built for): everything
imports, and the calls hand over their arguments through ctypes."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run(code, **env):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, env={**os.environ, **env}, capture_output=True, text=True,
                          timeout=600)


HIDE = "import sys; sys.modules['gemm_exl3_gemv_b200._binding'] = None\n"


def test_everything_imports_and_calls_go_through_ctypes():
    out = run(HIDE + """
from gemm_exl3_gemv_b200 import build
build.build()
from gemm_exl3_gemv_b200 import exl3 as ex, kvcache, stack
assert type(ex._binding).__name__ == "_CtypesBinding"
import pytest
sys.exit(pytest.main(["-q", "-p", "no:cacheprovider", "tests/test_abi_cache.py", "tests/test_abi.py", "-m", "not gpu"]))
""")
    assert out.returncode == 0, out.stdout[-3000:] + out.stderr[-2000:]


def test_the_build_leaves_the_compiled_binding_out_without_a_compiler(tmp_path):
    out = run(f"""
from gemm_exl3_gemv_b200 import build
build.BINDING = {str(tmp_path / "binding.so")!r}
build._compile_binding(True)
""", CC="no-such-compiler")
    assert out.returncode == 0 and "left out" in out.stderr and not os.listdir(tmp_path)


def test_the_compiled_binding_names_its_python():
    from gemm_exl3_gemv_b200 import build
    assert build.BINDING.endswith(".so") and sys.implementation.cache_tag.replace("-", "") in build.BINDING.replace("-", "")


@pytest.mark.gpu
def test_calls_on_the_gpu_through_ctypes():
    out = run(HIDE + """
import pytest
sys.exit(pytest.main(["-q", "-x", "-p", "no:cacheprovider", "tests/test_gpu_decode_step.py", "tests/test_gpu_q4.py",
                      "tests/test_gpu_kvcache.py", "tests/test_gpu_attention.py", "-k",
                      "serving or one_row or strided or truncate or compact or default or stack"]))
""")
    assert out.returncode == 0, out.stdout[-3000:] + out.stderr[-2000:]


def test_both_forms_take_numbers_of_other_kinds():
    """NumPy's whole numbers as Python's; a number with a fraction is none."""
    code = """
import numpy as np
from gemm_exl3_gemv_b200 import exl3 as ex
b = ex._binding
assert b.kv_extend(None, np.int64(1), np.int32(1), 17, None, 0) == ex.EXL3_ERR_INVALID_ARG
for args in ((None, 1.0, 1, 17, None, 0), (None, 1, 1, "17", None, 0), (None, None, 1, 17, None, 0)):
    try:
        b.kv_extend(*args)
    except TypeError:
        continue
    raise AssertionError(args)
print(type(b).__name__)
"""
    for first, kind in (("", "module"), (HIDE, "_CtypesBinding")):
        out = run(first + code)
        assert out.returncode == 0 and out.stdout.strip() == kind, out.stdout + out.stderr
