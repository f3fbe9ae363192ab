"""Calls of the attention and of cache writes that the documentation allows or
refuses: counts out of range, results in place of the queries."""
import numpy as np
import pytest

from test_gpu_attention import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    from gemm_exl3_gemv_b200 import exl3
    return exl3


@pytest.mark.parametrize("group", [2, 8])                    # both kernels
@pytest.mark.parametrize("bad", [-1, 5, 2 ** 31 - 1, -2 ** 31])
def test_counts_out_of_range_are_reported(ex, bad, group):
    """The entry's rows are left as they were, the others are right."""
    c = Case([300, 90, 1400], [4, 4, 2], m=4, group=group, page=64, seed=group)
    counts, q = list(c.counts), c.q
    c.counts = [4, bad, 2]
    out, lse = c.run()
    assert c.cache.status() == ex.EXL3_ERR_INDEX
    assert (out[1] == 77).all() and (lse[1] == 77).all()
    for b in (0, 2):
        c.seqs, c.counts, c.q = [b], [counts[b]], q[b:b + 1]
        c.check((out[b:b + 1], lse[b:b + 1]))


@pytest.mark.parametrize("bad", [-1, 4, -2 ** 31])
def test_writes_of_bad_counts_change_nothing(ex, bad):
    import torch
    c = Case([300, 90], [1, 1], page=64)
    before = c.cache.k.view(torch.int16).clone()
    kv = torch.ones(2, 3, 2, 128, dtype=torch.float16, device="cuda")
    c.cache.write(0, c.ids([0, 1]), kv, kv, counts=c.ids([2, bad]))
    assert c.cache.status() == ex.EXL3_ERR_INDEX
    assert torch.equal(c.cache.k.view(torch.int16), before)


@pytest.mark.parametrize("m,group,lens", [(1, 4, [90, 700, 3]), (3, 5, [9000, 40, 900]), (16, 5, [5000, 800, 333]), (32, 8, [2500, 64, 32])])
def test_results_in_place_of_the_queries(ex, m, group, lens):
    """Short sequences, and long ones that several CTAs share and either kernel joins: the same bits."""
    import torch
    c = Case(lens, [m, m, max(1, m - 1)], kv_heads=2, group=group, dim=128, page=64, m=m, seed=m)
    q, seqs, counts = torch.from_numpy(c.q).cuda(), c.ids(c.seqs), c.ids(c.counts)
    want = c.cache.attention(0, seqs, q, counts=counts)
    for _ in range(5):
        x = q.clone()
        assert c.cache.attention(0, seqs, x, counts=counts, out=x).data_ptr() == x.data_ptr()
        for b, n in enumerate(c.counts):
            assert torch.equal(x[b, :n], want[b, :n]) and torch.equal(x[b, n:], q[b, n:])
