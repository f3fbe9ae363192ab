"""Run by tests/test_gpu_debug_bounds_q4.py in a fresh process whose binding
loads the debug-bounds build: 4-bit products of every kernel, shape and cut,
each checked against the definition in fp64, with a clean status word."""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import numpy as np  # noqa: E402
import torch  # noqa: E402

from gemm_exl3_gemv_b200 import exl3 as ex  # noqa: E402
from test_gpu_q4 import close, make, reference  # noqa: E402


def main():
    assert ex.LIB_PATH.endswith("libexl3_debug.so"), ex.LIB_PATH
    n = 0
    for m in (1, 2, 7, 8, 9, 16, 17, 24, 25, 32):
        for k, n_out, group in ((64, 16, 64), (192, 80, 32), (1088, 144, 64), (640, 384, 128), (8192, 64, 32), (5120, 1024, 128),
                                (2048, 4112, 64)):
            for fp32 in (True, False):
                c = make(m, k, n_out, group, seed=m + k, zero=(m + k) % 3 != 0)
                d = {x: torch.from_numpy(a).cuda() for x, a in c.items() if isinstance(a, np.ndarray)}
                ws = torch.zeros(int(ex.lib.exl3_q4_workspace_bytes(m, k, n_out)), dtype=torch.uint8, device="cuda")
                y = ex.q4_gemm(d["x"], ex.q4_pack(d["q"]), d["scale"], d.get("zero"), group, fp32=fp32, workspace=ws)
                assert ex.workspace_status(ws) == ex.EXL3_OK, (m, k, n_out, group)
                close(y, *reference(c), fp32)
                n += 1
    print(f"debug-bounds 4-bit cases ok: {n}")


if __name__ == "__main__":
    main()
