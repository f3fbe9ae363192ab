"""Attention whose copies are all withheld (the workspace's injection word), in
CTAs that take many sequences one after the other: every wait is bounded, all
warps of a CTA leave together, the status says so, and with the workspace
cleared the next call is right."""
import numpy as np
import pytest

from test_gpu_attention import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    from gemm_exl3_gemv_b200 import exl3
    return exl3


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("m,group,window,sinks", [(1, 3, 0, 0), (2, 8, 40, 3), (5, 4, 0, 0), (9, 4, 70, 5), (32, 8, 0, 0)])
def test_many_short_sequences_in_a_cta(ex, dim, m, group, window, sinks):
    """700 or 160 sequences of one to four tiles and two heads: several times the GPU's CTAs, so that each takes
    many stretches, most of them of tiles that not every row sees."""
    rng = np.random.default_rng(m + dim)
    n = 700 if m < 32 else 160
    lens = rng.integers(m, 200, n).tolist()
    c = Case(lens, rng.integers(0, m + 1, n).tolist(), kv_heads=2, group=group, dim=dim, page=32, m=m, seed=m)
    ws = c.cache.attention_workspace(n, m, 2 * group)
    ws[4:8] = 1
    c.run(window=window, sinks=sinks, workspace=ws)
    assert ex.workspace_status(ws) == ex.EXL3_ERR_TIMEOUT
    ws.zero_()
    c.check(c.run(window=window, sinks=sinks, workspace=ws), window=window, sinks=sinks)
    assert ex.workspace_status(ws) == ex.EXL3_OK


@pytest.mark.parametrize("m", [1, 8])
def test_cut_sequences_with_a_second_kernel(ex, m):
    """A few long sequences beside short ones: the parts of cut sequences go on the second kernel's list whatever
    they hold."""
    c = Case([9000, 40, 70, 6000, 3], [m, m, m, m, min(m, 3)], kv_heads=1, group=5, dim=128, page=64, m=m, seed=3)
    assert c.cache.attention_launches(5, m, 5) == 2
    ws = c.cache.attention_workspace(5, m, 5)
    ws[4:8] = 1
    c.run(workspace=ws)
    assert ex.workspace_status(ws) == ex.EXL3_ERR_TIMEOUT
    ws.zero_()
    c.check(c.run(workspace=ws))
    assert ex.workspace_status(ws) == ex.EXL3_OK


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("m,group", [(1, 4), (6, 4)])        # both kernels
@pytest.mark.parametrize("v", [2, 8])
def test_some_tiles_come_and_the_others_do_not(ex, m, group, v, dim):
    """The first v - 1 tiles of each CTA arrive, so that products are done and stages in use when a wait runs out."""
    c = Case([64 * 70 * 9, 1000, 64 * 70 * 5], [m] * 3, kv_heads=4, group=group, dim=dim, page=64, m=m, seed=v)
    ws = c.cache.attention_workspace(3, m, 4 * group)
    ws[4:8] = c.torch.tensor([v, 0, 0, 0], dtype=c.torch.uint8)
    c.run(workspace=ws)
    assert ex.workspace_status(ws) == ex.EXL3_ERR_TIMEOUT
    ws.zero_()
    c.check(c.run(workspace=ws))
    assert ex.workspace_status(ws) == ex.EXL3_OK
