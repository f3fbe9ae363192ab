"""The paged cache's calls on the GPU against a plain model: every table entry,
length, reference count, free bit, key and value."""
import numpy as np
import pytest

from cache_model import CacheModel

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    from gemm_exl3_gemv_b200 import exl3
    return exl3


class Pair:
    """A cache on the GPU and its model, driven by the same calls."""

    def __init__(self, layers=2, pages=40, heads=2, page_size=16, dim=64, seqs=8, max_pages=6, seed=0):
        import torch
        from gemm_exl3_gemv_b200.kvcache import KvCache
        self.torch = torch
        self.rng = np.random.default_rng(seed)
        self.gpu = KvCache.empty(layers, pages, heads, page_size, dim, seqs, max_pages)
        self.model = CacheModel(layers, pages, heads, page_size, dim, seqs, max_pages)

    def ids(self, values):
        return self.torch.tensor(list(values), dtype=self.torch.int32, device="cuda")

    def grow(self, seqs, counts, m=None):
        """extend and write in every layer; False if the model refuses."""
        torch, mod = self.torch, self.model
        m = m or max(counts)
        layers, _, heads, _, dim = mod.k.shape
        self.gpu.extend(self.ids(seqs), m, counts=self.ids(counts))
        ok = mod.extend(seqs, counts)
        for layer in range(layers):
            k = self.rng.standard_normal((len(seqs), m, heads, dim)).astype(np.float16)
            v = self.rng.standard_normal((len(seqs), m, heads, dim)).astype(np.float16)
            if ok:
                mod.write(layer, seqs, counts, k, v)
            self.gpu.write(layer, self.ids(seqs), torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), counts=self.ids(counts))
        return ok

    def check(self, status=0):
        assert self.gpu.status() == status
        m = self.model
        assert self.gpu.lens.tolist() == m.lens
        assert self.gpu.refs.tolist() == m.refs
        assert np.array_equal(self.gpu.free.cpu().numpy().view(np.uint32), m.free_words())
        assert np.array_equal(self.gpu.table.cpu().numpy(), m.full_table(m.max_pages))
        for mine, theirs in ((self.gpu.k, m.k), (self.gpu.v, m.v)):
            assert np.array_equal(mine.cpu().numpy().view(np.uint16), theirs.view(np.uint16))


def test_reset_and_empty_lists(ex):
    p = Pair(pages=33)
    p.check()
    none = p.ids([])
    p.gpu.extend(none, 3)
    p.gpu.truncate(none)
    p.gpu.fork(none, none)
    p.gpu.compact()
    p.check()
    p.grow([1, 3], [5, 17])
    p.check()
    p.gpu.reset()
    p.model.__init__(*p.model.k.shape, 8, 6)
    p.model.k[:], p.model.v[:] = p.gpu.k.cpu().numpy(), p.gpu.v.cpu().numpy()
    p.check()


@pytest.mark.parametrize("page_size,dim,heads", [(16, 64, 1), (32, 128, 3), (64, 64, 2), (128, 128, 1), (256, 64, 2)])
def test_grow_in_pieces(ex, page_size, dim, heads):
    """Tokens one by one, across page borders, whole pages at once, none."""
    p = Pair(pages=30, heads=heads, page_size=page_size, dim=dim, max_pages=5, seed=page_size)
    for seqs, counts in [([0], [1]), ([0, 2], [page_size - 1, page_size]), ([2, 0, 5], [0, 1, page_size + 1]),
                         ([5, 2], [2 * page_size, 3]), ([7], [5 * page_size])]:
        assert p.grow(seqs, counts)
        p.check()


def test_counts_default_to_all(ex):
    p = Pair()
    import torch
    p.gpu.extend(p.ids([4, 1]), 7)
    p.model.extend([4, 1], [7, 7])
    kv = np.random.default_rng(1).standard_normal((2, 2, 7, 2, 64)).astype(np.float16)
    p.gpu.write(1, p.ids([4, 1]), torch.from_numpy(kv[0]).cuda(), torch.from_numpy(kv[1]).cuda())
    p.model.write(1, [4, 1], [7, 7], kv[0], kv[1])
    p.check()


def test_write_takes_strided_rows(ex):
    """Keys and values as parts of one projection's output rows, of a batch padded behind."""
    import torch
    p = Pair(heads=2, dim=64)
    wide = torch.randn(3, 9, 640, device="cuda", dtype=torch.float16)
    k = wide[:, :5, 256:384].view(3, 5, 2, 64)
    v = wide[:, :5, 384:512].view(3, 5, 2, 64)
    counts = [5, 2, 4]
    p.gpu.extend(p.ids([0, 6, 3]), 5, counts=p.ids(counts))
    p.model.extend([0, 6, 3], counts)
    p.gpu.write(0, p.ids([0, 6, 3]), k, v, counts=p.ids(counts))
    p.model.write(0, [0, 6, 3], counts, k.cpu().numpy(), v.cpu().numpy())
    p.check()


def test_truncate_fork_free(ex):
    p = Pair(pages=60, max_pages=8)
    p.grow([0, 1, 2], [50, 33, 100])
    for seqs, lens in [([1, 0], [32, 200]), ([2], [97]), ([2], [96]), ([0], [49]), ([1], [0]), ([1], [5])]:
        p.gpu.truncate(p.ids(seqs), p.ids(lens))
        p.model.truncate(seqs, lens)
        p.check()
    # one source several times, an empty source
    p.gpu.fork(p.ids([2, 2, 0, 1]), p.ids([5, 3, 7, 6]))
    p.model.fork([2, 2, 0, 1], [5, 3, 7, 6])
    p.check()
    # the first of several holders to grow, all of them at once, and a holder whose last page is full
    p.grow([7], [1])
    p.check()
    p.grow([0, 7], [3, 2])
    p.check()
    p.grow([5, 2, 3], [1, 1, 1])
    p.check()
    p.gpu.truncate(p.ids([2, 5]))
    p.model.truncate([2, 5], [0, 0])
    p.check()


def test_all_holders_of_a_part_page_grow_at_once(ex):
    """Each gets a copy; the page itself is free afterwards."""
    p = Pair(pages=20)
    p.grow([0], [21])
    p.gpu.fork(p.ids([0, 0]), p.ids([1, 2]))
    p.model.fork([0, 0], [1, 2])
    p.grow([2, 0, 1], [1, 20, 2])
    assert p.model.refs[1] == 0
    p.check()


def test_compact(ex):
    p = Pair(pages=50, max_pages=8, seqs=9)
    p.gpu.compact()
    p.check()
    p.grow([0, 1, 2, 3, 4], [40, 100, 1, 64, 90])
    p.gpu.fork(p.ids([4]), p.ids([8]))
    p.model.fork([4], [8])
    p.gpu.compact()
    p.model.compact()
    p.check()
    for gone in ([1], [0, 3], [2, 8]):
        p.gpu.truncate(p.ids(gone))
        p.model.truncate(gone, [0] * len(gone))
        p.gpu.compact()
        p.model.compact()
        p.check()
        p.grow([gone[0], 4], [20, 1])
        p.check()


def test_long_random_run(ex):
    """Hundreds of calls of every kind on one cache, with refusals for want of pages among them."""
    p = Pair(layers=1, pages=70, heads=1, page_size=16, seqs=20, max_pages=12, seed=11)
    rng, refused = np.random.default_rng(5), 0
    for step in range(250):
        kind = rng.integers(0, 10)
        some = rng.permutation(20)[:rng.integers(1, 8)].tolist()
        if kind < 5:
            ok = p.grow(some, rng.integers(0, 40, len(some)).tolist(), m=40)
            if not ok:
                refused += 1
                p.check(ex.EXL3_ERR_CACHE_FULL)
        elif kind < 8:
            lens = rng.integers(0, 150, len(some)).tolist()
            p.gpu.truncate(p.ids(some), p.ids(lens))
            p.model.truncate(some, lens)
        elif kind == 8:
            dst = [s for s in range(20) if p.model.lens[s] == 0][:3]
            src = [s for s in range(20) if p.model.lens[s] > 0]
            if dst and src:
                src = [src[i % len(src)] for i in range(len(dst))]
                p.gpu.fork(p.ids(src), p.ids(dst))
                p.model.fork(src, dst)
        else:
            p.gpu.compact()
            p.model.compact()
        if step % 10 == 0:
            p.check()
    p.check()
    assert refused > 3


def test_large_pool_and_long_lists(ex):
    """A thousand sequences in one list, tens of thousands of pages."""
    n = 1024
    p = Pair(layers=1, pages=40000, heads=1, page_size=16, dim=64, seqs=1500, max_pages=40, seed=3)
    order = np.random.default_rng(2).permutation(1500)[:n]
    counts = np.random.default_rng(3).integers(0, 300, n)
    p.gpu.extend(p.ids(order), 300, counts=p.ids(counts))
    p.model.extend(order.tolist(), counts.tolist())
    p.check()
    p.gpu.truncate(p.ids(order[::2]))
    p.model.truncate(order[::2].tolist(), [0] * (n // 2))
    p.gpu.compact()
    p.model.compact()
    p.check()


def test_refused_steps_change_nothing(ex):
    """Lists with a bad or repeated number, too few pages, too few table entries: the call and the writes
    behind it do nothing until the status has been read."""
    p = Pair(pages=10, seqs=4, max_pages=6)
    p.grow([0, 1], [20, 30])
    p.check()
    import torch
    kv = torch.ones(2, 9, 2, 64, dtype=torch.float16, device="cuda")

    def refused(call, status):
        call()
        p.gpu.write(0, p.ids([0, 1]), kv, kv)
        p.gpu.extend(p.ids([2]), 1)
        p.check(status)

    idx, full = ex.EXL3_ERR_INDEX, ex.EXL3_ERR_CACHE_FULL
    refused(lambda: p.gpu.extend(p.ids([0, 4]), 9), idx)
    refused(lambda: p.gpu.extend(p.ids([0, -1]), 9), idx)
    refused(lambda: p.gpu.extend(p.ids([1, 0, 1]), 9), idx)
    refused(lambda: p.gpu.extend(p.ids([1, 0]), 9, counts=p.ids([3, 10])), idx)
    refused(lambda: p.gpu.extend(p.ids([1, 0]), 9, counts=p.ids([3, -1])), idx)
    refused(lambda: p.gpu.extend(p.ids([3, 2]), 60), full)            # 8 pages, 6 are free
    refused(lambda: p.gpu.extend(p.ids([0]), 77), full)               # 97 tokens, a table row holds 96
    refused(lambda: p.gpu.truncate(p.ids([0, 0])), idx)
    refused(lambda: p.gpu.truncate(p.ids([0, 7])), idx)
    refused(lambda: p.gpu.truncate(p.ids([0, 1]), p.ids([3, -2])), idx)
    refused(lambda: p.gpu.fork(p.ids([0, 1]), p.ids([2, 2])), idx)
    refused(lambda: p.gpu.fork(p.ids([0, 1]), p.ids([2, 0])), idx)
    refused(lambda: p.gpu.fork(p.ids([0, 9]), p.ids([2, 3])), idx)
    # a pair whose destination holds tokens is left out, the others are not
    p.gpu.fork(p.ids([0, 0]), p.ids([1, 2]))
    p.model.fork([0], [2])
    p.check(idx)
    # and the cache goes on
    assert p.grow([0, 3], [5, 16])
    p.check()


def test_refused_writes_change_nothing(ex):
    """A write by itself, with a bad or repeated number, or more tokens than rows."""
    import torch
    p = Pair(pages=10, seqs=4, max_pages=6)
    p.grow([0, 1], [20, 30])
    kv = torch.ones(2, 9, 2, 64, dtype=torch.float16, device="cuda")
    for seqs, counts in (([0, 4], None), ([-1, 0], None), ([1, 1], None), ([0, 0], [1, 0]), ([1, 0], [3, 10]),
                         ([0, 2 ** 31 - 1], None)):
        p.gpu.write(1, p.ids(seqs), kv, kv, counts=None if counts is None else p.ids(counts))
        p.check(ex.EXL3_ERR_INDEX)


def test_offsets_past_32_bits(ex):
    """A pool of 2.5e9 elements (5 GB) of keys: sequences whose pages lie at its end are grown, forked, copied
    and written, attended to, moved to its front by a compaction, and attended to again."""
    import torch
    import cache_model
    from gemm_exl3_gemv_b200.kvcache import KvCache
    heads, ps, dim, pages = 8, 64, 128, 38400
    ids = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    c = KvCache.empty(1, pages, heads, ps, dim, 3, pages)
    assert c.k.numel() > 2 ** 31
    c.extend(ids(0), (pages - 8) * ps)
    rng = np.random.default_rng(5)
    new = lambda m: rng.standard_normal((1, m, heads, dim)).astype(np.float16)
    dev = lambda a: torch.from_numpy(a).cuda()
    k1, v1, k2, v2, q = new(100), new(100), new(70), new(70), rng.standard_normal((2, 3, 16, dim)).astype(np.float16)
    c.extend(ids(1), 100)
    c.write(0, ids(1), dev(k1), dev(v1))
    c.fork(ids(1), ids(2))
    c.extend(ids(2), 70)                                      # its last page is copied
    c.write(0, ids(2), dev(k2), dev(v2))
    assert c.table[1, :2].tolist() == [pages - 8, pages - 7] and c.table[2, :3].tolist() == [pages - 8, pages - 6, pages - 5]
    out = c.attention(0, ids(1, 2), dev(q))
    cat = lambda a, b: np.concatenate([a[0], b[0]]).astype(np.float64)
    for b, (k, v) in enumerate(((k1[0].astype(np.float64), v1[0].astype(np.float64)), (cat(k1, k2), cat(v1, v2)))):
        ref, _, tol, _ = cache_model.attention(q[b].astype(np.float64), k, v, len(k) - 3, dim ** -0.5)
        assert np.all(np.abs(out[b].double().cpu().numpy() - ref) <= tol)
    c.truncate(ids(0))
    c.compact()
    assert c.table[1, :2].tolist() == [0, 1] and c.table[2, :3].tolist() == [0, 2, 3]
    assert torch.equal(c.attention(0, ids(1, 2), dev(q)), out)
    c.check()


def test_repeated_status_reads_and_exception(ex):
    p = Pair()
    p.gpu.extend(p.ids([99]), 1)
    with pytest.raises(ex.Exl3Error) as e:
        p.gpu.check()
    assert e.value.status == ex.EXL3_ERR_INDEX
    p.gpu.check()


def test_bad_table_entries_are_not_followed(ex):
    """A page number out of range in the table: nothing is written there, the status says so."""
    import torch
    p = Pair(pages=10, seqs=4, max_pages=6)
    p.grow([0, 1], [20, 30])
    before = p.gpu.k.clone()
    good = p.gpu.table.clone()
    for bad in (-1, 10, 2 ** 30):
        p.gpu.table[0, 1] = bad
        kv = torch.ones(1, 2, 2, 64, dtype=torch.float16, device="cuda")
        p.gpu.write(0, p.ids([0]), kv, kv)
        assert p.gpu.status() == ex.EXL3_ERR_INDEX
        p.gpu.extend(p.ids([0]), 2)
        assert p.gpu.status() == ex.EXL3_ERR_INDEX
        p.gpu.table.copy_(good)
        assert torch.equal(before, p.gpu.k)
        p.check()


def test_captured_step_allocates_on_replay(ex):
    """A graph of one step grows the sequences at every replay, as the calls themselves do."""
    import torch
    p = Pair(pages=60, seqs=6, max_pages=10)
    p.grow([0, 2, 5], [15, 3, 30])
    p.gpu.fork(p.ids([5]), p.ids([1]))
    p.model.fork([5], [1])
    seqs, counts = p.ids([2, 1, 5, 0]), p.ids([3, 1, 2, 3])
    kv = torch.randn(2, 4, 3, 2, 64, device="cuda", dtype=torch.float16)
    back = p.ids([0])

    def step():
        p.gpu.extend(seqs, 3, counts=counts)
        for layer in range(2):
            p.gpu.write(layer, seqs, kv[layer], kv[1 - layer], counts=counts)
        p.gpu.truncate(back, cut)
        p.gpu.compact()

    cut = p.ids([17])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(5):
        kv.normal_()
        g.replay()
        assert p.model.extend([2, 1, 5, 0], [3, 1, 2, 3])
        a = kv.cpu().numpy()
        for layer in range(2):
            p.model.write(layer, [2, 1, 5, 0], [3, 1, 2, 3], a[layer], a[1 - layer])
        p.model.truncate([0], [17])
        p.model.compact()
        p.check()
    del g


def test_refusals_on_the_host(ex):
    import torch
    from gemm_exl3_gemv_b200.kvcache import KvCache
    p = Pair()
    seqs = p.ids([0, 1])
    rows = torch.zeros(2, 3, 2, 64, dtype=torch.float16, device="cuda")
    for call in (lambda: p.gpu.extend(seqs.long(), 1), lambda: p.gpu.extend(seqs.cpu(), 1),
                 lambda: p.gpu.extend(seqs, 1, counts=seqs[:1]), lambda: p.gpu.fork(seqs, seqs[:1]),
                 lambda: p.gpu.truncate(seqs, seqs.float()), lambda: p.gpu.write(0, seqs, rows.float(), rows),
                 lambda: p.gpu.write(0, seqs, rows[:, :, :1], rows[:, :, :1]),
                 lambda: p.gpu.write(0, seqs, rows, rows[:, :2]),
                 lambda: p.gpu.write(0, seqs, rows.transpose(1, 2).contiguous().transpose(1, 2), rows),
                 lambda: p.gpu.write(0, seqs, rows.cpu(), rows.cpu())):
        with pytest.raises(ValueError):
            call()
    for call, status in ((lambda: p.gpu.extend(seqs, 0), ex.EXL3_ERR_INVALID_ARG),
                         (lambda: p.gpu.write(2, seqs, rows, rows), ex.EXL3_ERR_INVALID_ARG),
                         (lambda: p.gpu.write(-1, seqs, rows, rows), ex.EXL3_ERR_INVALID_ARG),
                         (lambda: p.gpu.extend(torch.zeros(1025, dtype=torch.int32, device="cuda"), 1), ex.EXL3_ERR_UNSUPPORTED),
                         (lambda: KvCache.empty(1, 4, 1, 24, 64, 2, 2), ex.EXL3_ERR_UNSUPPORTED),
                         (lambda: KvCache.empty(1, 4, 1, 16, 96, 2, 2), ex.EXL3_ERR_UNSUPPORTED)):
        with pytest.raises(ex.Exl3Error) as e:
            call()
        assert e.value.status == status
    p.check()
