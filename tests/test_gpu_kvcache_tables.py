"""A cache made from a caller's own tensors, whose table rows hold other numbers
than -1 behind each sequence's last page: what stands there does not matter."""
import numpy as np
import pytest

from cache_model import CacheModel

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    from gemm_exl3_gemv_b200 import exl3
    return exl3


@pytest.mark.parametrize("layers,heads", [(1, 1), (4, 8)])
def test_numbers_behind_the_last_page_do_not_matter(ex, layers, heads):
    """Behind its last page every row names a page that several sequences hold.  Growth with and without copies
    of shared pages, again and again: bookkeeping, keys and values as in the model, nothing counted and left."""
    import torch
    from gemm_exl3_gemv_b200.kvcache import KvCache
    n, ps, dim, max_pages, pages = 120, 16, 64, 12, 1600
    rng = np.random.default_rng(layers)
    mod = CacheModel(layers, pages, heads, ps, dim, 2 * n, max_pages)
    mod.k[:] = rng.standard_normal(mod.k.shape).astype(np.float16)
    mod.v[:] = rng.standard_normal(mod.v.shape).astype(np.float16)
    assert mod.extend(list(range(n)), rng.integers(1, 60, n).tolist())
    mod.fork(list(range(0, n, 2)), list(range(n, n + n // 2)))
    shared = mod.table[0][0]
    assert mod.refs[shared] > 1
    table = np.array([row + [shared] * (max_pages - len(row)) for row in mod.table], np.int32)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    gpu = KvCache(dev(mod.k), dev(mod.v), dev(table), dev(np.array(mod.lens, np.int32)), dev(np.array(mod.refs, np.int32)),
                  dev(mod.free_words().view(np.int32)))

    def check():
        gpu.check()
        assert gpu.lens.tolist() == mod.lens and gpu.refs.tolist() == mod.refs
        assert np.array_equal(gpu.free.cpu().numpy().view(np.uint32), mod.free_words())
        got = gpu.table.cpu().numpy()
        for s, row in enumerate(mod.table):
            assert got[s, :len(row)].tolist() == row, s
        for mine, theirs in ((gpu.k, mod.k), (gpu.v, mod.v)):
            assert np.array_equal(mine.cpu().numpy().view(np.uint16), theirs.view(np.uint16))
        assert gpu.scratch.view(torch.int32)[:4].tolist()[:2] == [0, 0]

    check()
    for step in range(12):
        # odd steps: sequences that share nothing; even ones: some that do, too
        ids = rng.permutation(np.arange(1, n, 2) if step % 2 else np.arange(n + n // 2))[:40].tolist()
        counts = rng.integers(0, 17, len(ids)).tolist()
        counts = [min(c, max_pages * ps - mod.lens[s]) for s, c in zip(ids, counts)]
        gpu.extend(dev(np.array(ids, np.int32)), 17, counts=dev(np.array(counts, np.int32)))
        assert mod.extend(ids, counts)
        check()
    gpu.compact()
    mod.compact()
    check()
