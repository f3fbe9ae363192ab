"""4-bit products on tcgen05 whose inputs stop coming part-way (the workspace's
injection word): every wait is bounded, the status says so, and the next call is
right."""
import numpy as np
import pytest

from test_gpu_q4 import close, make, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    from gemm_exl3_gemv_b200 import exl3
    return exl3


# clusters of four, of three and none; more stages than the rings have places, and fewer; half a stage at the end
@pytest.mark.parametrize("m,k,n,group", [(32, 8192, 256, 128), (12, 6464, 6144, 64), (25, 5120, 19200, 32), (16, 1600, 256, 64)])
@pytest.mark.parametrize("v", [2, 7])
def test_some_stages_come_and_the_others_do_not(ex, m, k, n, group, v):
    import torch
    c = make(m, k, n, group, seed=v)
    d = {k: torch.from_numpy(a).cuda() for k, a in c.items() if isinstance(a, np.ndarray)}
    packed, ws = ex.q4_pack(d["q"]), ex.q4_alloc_workspace(m, k, n)
    ws[4:8] = torch.tensor([v, 0, 0, 0], dtype=torch.uint8)
    ex.q4_gemm(d["x"], packed, d["scale"], d["zero"], group, workspace=ws)
    stages = -(-k // 128)
    blocks = -(-n // 128)
    splits = max(1, min(4, 148 // blocks, stages))
    held_back = stages // splits + (stages % splits > 0) > v - 1      # of the CTA with the most stages
    assert ex.workspace_status(ws) == (ex.EXL3_ERR_TIMEOUT if held_back else ex.EXL3_OK)
    ws[4:8] = 0
    close(ex.q4_gemm(d["x"], packed, d["scale"], d["zero"], group, fp32=True, workspace=ws), *reference(c), True)
    assert ex.workspace_status(ws) == ex.EXL3_OK
