"""exl3_paged_attention on the GPU against an fp64 evaluation of the definition
(cache_model.attention, which also derives the error allowed)."""
import numpy as np
import pytest

import cache_model

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    from gemm_exl3_gemv_b200 import exl3
    return exl3


class Case:
    """Sequences of the given lengths on scattered pages, queries for their last tokens.  Memory that holds
    no token is NaN."""

    def __init__(self, lens, counts, kv_heads=2, group=3, dim=128, page=16, m=None, seed=0, layers=1, spread=1.0, spare=5):
        import torch
        from gemm_exl3_gemv_b200.kvcache import KvCache
        self.torch, rng = torch, np.random.default_rng(seed)
        need = [-(-n // page) for n in lens]
        n_pages = sum(need) + spare
        shape = (layers, n_pages, kv_heads, page, dim)
        self.k, self.v = np.full(shape, np.nan, np.float16), np.full(shape, np.nan, np.float16)
        order = rng.permutation(n_pages).tolist()
        table = np.full((len(lens), max(max(need), 1) + 2), -1, np.int32)
        refs = np.zeros(n_pages, np.int32)
        self.tokens = []                              # per sequence: keys, values (layers, tokens, heads, dim)
        for s, n in enumerate(lens):
            mine = [order.pop() for _ in range(need[s])]
            table[s, :need[s]] = mine
            refs[mine] = 1
            kv = rng.standard_normal((2, layers, n, kv_heads, dim)).astype(np.float16)
            kv[0] *= spread
            for t in range(n):
                self.k[:, mine[t // page], :, t % page] = kv[0][:, t]
                self.v[:, mine[t // page], :, t % page] = kv[1][:, t]
            self.tokens.append(kv)
        self.lens, self.counts, self.page = list(lens), list(counts), page
        self.m = m or max(max(counts), 1)
        self.q = rng.standard_normal((len(lens), self.m, kv_heads * group, dim)).astype(np.float16)
        dev = lambda a: torch.from_numpy(a).cuda()
        self.cache = KvCache(dev(self.k), dev(self.v), dev(table), dev(np.array(lens, np.int32)), dev(refs),
                             torch.zeros((n_pages + 31) // 32, dtype=torch.int32, device="cuda"))
        self.seqs = list(range(len(lens)))
        self.scale = dim ** -0.5

    def ids(self, x):
        return self.torch.tensor(x, dtype=self.torch.int32, device="cuda")

    def run(self, layer=0, **kw):
        torch = self.torch
        out = torch.full(self.q.shape, 77.0, dtype=torch.float16, device="cuda")
        lse = torch.full(self.q.shape[:3], 77.0, dtype=torch.float32, device="cuda")
        self.cache.attention(layer, self.ids(self.seqs), torch.from_numpy(self.q).cuda(), counts=self.ids(self.counts),
                             out=out, lse=lse, **kw)
        return out, lse

    def check(self, got, layer=0, window=0, sinks=0, scale=None):
        out, lse = (x.double().cpu().numpy() for x in got)
        for b, (s, c) in enumerate(zip(self.seqs, self.counts)):
            assert np.all(out[b, c:] == 77) and np.all(lse[b, c:] == 77), "rows behind the last were touched"
            if c == 0:
                continue
            k, v = (x[layer].astype(np.float64) for x in self.tokens[s])
            ref, rl, ot, lt = cache_model.attention(self.q[b, :c].astype(np.float64), k, v, self.lens[s] - c,
                                                    self.scale if scale is None else scale, window, sinks)
            assert np.all(np.abs(out[b, :c] - ref) <= ot), (b, np.nanmax(np.abs(out[b, :c] - ref) / ot))
            none = np.isinf(rl)
            assert np.all(lse[b, :c][none] == -np.inf)
            assert np.all(np.abs(lse[b, :c] - rl)[~none] <= lt[~none]), b
        assert self.cache.status() == 0


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_decode_lengths(ex, dim, page):
    """One token of each sequence: every kind of tail of a page and of a tile, one token in all."""
    c = Case([1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300, 511, 512, 513], [1] * 15, dim=dim, page=page, seed=page)
    c.check(c.run())


@pytest.mark.parametrize("kv_heads,group", [(1, 1), (8, 5), (2, 8), (1, 16), (3, 17), (1, 32)])
@pytest.mark.parametrize("m", [1, 2, 3, 6, 13, 16, 31, 32])
def test_heads_and_rows(ex, kv_heads, group, m):
    """Row counts on both sides of every row tile, causal among the new tokens, ragged counts with none among them."""
    rng = np.random.default_rng(m)
    lens = [m, m + 1, 70 + m, 200]
    counts = [m, int(rng.integers(1, m + 1)), 0, m]
    c = Case(lens, counts, kv_heads=kv_heads, group=group, dim=64 if group % 2 else 128, page=32, m=m, seed=m + group)
    c.check(c.run())


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 3), (64, 0), (64, 4), (65, 64), (100, 65), (128, 130),
                                          (1000, 5), (5, 1000), (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("m", [1, 9])
def test_window_and_sinks(ex, window, sinks, m):
    c = Case([m, 40, 64 + m, 130, 333, 700], [m, min(m, 40), m, m, m, m], dim=64, page=16, m=m, group=2, seed=window % 97)
    c.check(c.run(window=window, sinks=sinks), window=window, sinks=sinks)


def test_long_sequences_are_split_and_joined(ex):
    c = Case([9001, 3, 20011], [1, 1, 1], kv_heads=2, group=2, dim=64, page=64, seed=1)
    c.check(c.run())
    c = Case([6000], [20], kv_heads=1, group=3, dim=128, page=128, seed=2)
    c.check(c.run())


def test_many_sequences(ex):
    rng = np.random.default_rng(4)
    lens = rng.integers(1, 60, 500).tolist()
    c = Case(lens, [1] * 500, kv_heads=1, group=2, dim=64, page=16, seed=4)
    c.seqs = rng.permutation(500).tolist()
    c.check(c.run())


def test_large_scores_and_other_scales(ex):
    """Scores of hundreds: the running maximum keeps every exponential in range."""
    c = Case([700, 33], [1, 2], dim=128, spread=30.0, seed=6, m=2)
    c.check(c.run())
    for scale in (0.0, -0.05, 1e-6):
        c = Case([200, 33], [1, 2], dim=64, seed=7, m=2)
        c.check(c.run(scale=scale), scale=scale)


@pytest.mark.parametrize("group", [2, 3])                    # 12 and 18 rows: both kernels
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan"), 65504.0])
def test_unseen_tokens_do_not_matter(ex, value, group):
    """Keys and values that are not finite, in tokens that a row does not see: later drafted tokens, tokens
    outside the window.  The rows that do see one get what the formula gives (not a finite number)."""
    import torch
    m, window, sinks = 6, 40, 2
    c = Case([100, 170], [m, m], dim=64, page=32, m=m, group=group, seed=8)
    seen_by = {}
    for s, n in enumerate(c.lens):
        for t in (n - 2, n - m, 3, n - m - window):          # late draft, first draft, never seen, just out of the first row
            c.tokens[s][1][:, t, :, 5] = value               # a value element
            seen_by.setdefault(s, []).append(t)
    for s, n in enumerate(c.lens):
        for t in range(n):
            page = int(c.cache.table[s, t // c.page])
            c.cache.v[:, page, :, t % c.page] = torch.from_numpy(c.tokens[s][1][:, t]).cuda()
    out, _ = c.run(window=window, sinks=sinks)
    out = out.double().cpu().numpy()
    for s, n in enumerate(c.lens):
        k, v = (x[0].astype(np.float64) for x in c.tokens[s])
        for i in range(m):
            p = n - m + i
            see = cache_model.visible(p, n, window, sinks)
            touched = any(see[t] for t in seen_by[s])
            vv = np.where(see[:, None, None], v, 0.0)
            if touched and not np.isfinite(value):
                assert np.all(~np.isfinite(out[s, i, :, 5])), (s, i)
                vv[:, :, 5] = 0.0
            ref, _, tol, _ = cache_model.attention(c.q[s, i:i + 1].astype(np.float64), k, vv, p, c.scale, window, sinks)
            cols = [x for x in range(64) if x != 5] if touched and not np.isfinite(value) else list(range(64))
            assert np.all(np.abs(out[s, i] - ref[0])[:, cols] <= tol[0][:, cols]), (s, i)


@pytest.mark.parametrize("dim,group", [(64, 3), (64, 8), (128, 4), (128, 32)])
def test_unseen_keys_do_not_matter(ex, dim, group):
    import torch
    m = 4
    c = Case([90, 130], [m, m], dim=dim, page=32, m=m, group=group, seed=9)
    first = c.run()[0].clone()
    for s, n in enumerate(c.lens):
        t = n - 1                                            # seen by the last row alone
        page = int(c.cache.table[s, t // c.page])
        c.cache.k[:, page, :, t % c.page] = float("nan")
        c.cache.v[:, page, :, t % c.page] = float("nan")
    got = c.run()[0]
    assert torch.equal(got[:, :m - 1], first[:, :m - 1])
    assert torch.isnan(got[:, m - 1]).all()


def test_more_new_tokens_than_tokens(ex):
    """A length below the count (a sequence that was never extended): rows before the first token see nothing."""
    import torch
    c = Case([2, 0, 50], [5, 3, 1], dim=64, m=5, seed=10)
    out, lse = c.run()
    assert (out[0, :3] == 0).all() and torch.isinf(lse[0, :3]).all()
    assert (out[1, :3] == 0).all() and torch.isinf(lse[1, :3]).all()
    k, v = (x[0].astype(np.float64) for x in c.tokens[0])
    ref, _, tol, _ = cache_model.attention(c.q[0, 3:5].astype(np.float64), k, v, 0, c.scale)
    assert np.all(np.abs(out[0, 3:5].double().cpu().numpy() - ref) <= tol)


def test_layers_strides_and_no_lse(ex):
    """Another layer; queries as part of a wider projection; results into a wider buffer; no lse."""
    import torch
    c = Case([30, 77], [3, 2], dim=64, group=2, kv_heads=2, m=3, layers=3, seed=11)
    wide = torch.randn(2, 5, 1000, dtype=torch.float16, device="cuda")
    q = wide[:, 1:4, 512:768].view(2, 3, 4, 64)
    c.q = q.cpu().numpy()
    into = torch.full((2, 4, 600), 77.0, dtype=torch.float16, device="cuda")
    out = into[:, :3, 64:320].view(2, 3, 4, 64)
    for layer in (2, 0):
        out.fill_(77.0)
        ret = c.cache.attention(layer, c.ids(c.seqs), q, counts=c.ids(c.counts), out=out)
        assert ret.data_ptr() == out.data_ptr()
        lse = c.run(layer)[1]
        c.check((out, lse), layer)
    assert (into[:, 3] == 77).all() and (into[:, :, :64] == 77).all() and (into[:, :, 320:] == 77).all()


def test_default_output_and_counts(ex):
    import torch
    c = Case([30, 77], [3, 3], dim=64, m=3, seed=12)
    q = torch.from_numpy(c.q).cuda()
    out = c.cache.attention(0, c.ids(c.seqs), q)
    assert torch.equal(out, c.run()[0])
    c.counts = [2, 0]
    out = c.cache.attention(0, c.ids(c.seqs), q, counts=c.ids(c.counts))
    assert (out[0, 2:] == 0).all() and (out[1] == 0).all()
    assert torch.equal(out[0, :2], c.run()[0][0, :2])
    assert c.cache.attention(0, c.ids([]), q[:0]).shape == (0, 3, 6, 64)


def test_repeatable_in_graphs_and_streams(ex):
    """Bitwise the same: call after call with one workspace, in two graphs that share it, on another stream;
    after other shapes used the workspace."""
    import torch
    c = Case([3000, 41, 700], [2, 2, 1], dim=128, page=64, m=2, seed=13)
    d = Case([200, 900], [16, 9], dim=128, page=64, m=16, seed=14)
    ws = d.cache.attention_workspace(2, 16, 6)
    first = [x.clone() for x in c.run(workspace=ws)]
    other = [x.clone() for x in d.run(workspace=ws)]
    c.check(first)
    d.check(other)
    same = lambda a, b: all(torch.equal(x, y) for x, y in zip(a, b))
    for _ in range(3):
        assert same(c.run(workspace=ws), first) and same(d.run(workspace=ws), other)
    qs, seqs, counts = torch.from_numpy(c.q).cuda(), c.ids(c.seqs), c.ids(c.counts)
    dq, dseqs, dcounts = torch.from_numpy(d.q).cuda(), d.ids(d.seqs), d.ids(d.counts)
    graphs = []
    o1, o2 = torch.empty_like(first[0]), torch.empty_like(other[0])
    for cache, s, q, n, out in ((c.cache, seqs, qs, counts, o1), (d.cache, dseqs, dq, dcounts, o2)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            cache.attention(0, s, q, counts=n, out=out, workspace=ws)
        graphs.append(g)
    for _ in range(3):
        o1.fill_(77.0), o2.fill_(77.0)
        for g in graphs:
            g.replay()
        assert torch.equal(o1, first[0]) and torch.equal(o2, other[0])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    o1.fill_(77.0)
    side.wait_stream(torch.cuda.current_stream())
    c.cache.attention(0, seqs, qs, counts=counts, out=o1, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(o1, first[0])
    assert ex.workspace_status(ws) == ex.EXL3_OK
    del graphs


def test_graph_follows_the_lengths(ex):
    """A captured call reads the lengths at every replay."""
    import torch
    c = Case([500, 64], [1, 1], dim=64, page=16, seed=15)
    q, seqs = torch.from_numpy(c.q).cuda(), c.ids(c.seqs)
    ws = c.cache.attention_workspace(2, 1, 6)
    out, lse = torch.empty(c.q.shape, dtype=torch.float16, device="cuda"), torch.empty(c.q.shape[:3], device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.cache.attention(0, seqs, q, out=out, lse=lse, workspace=ws)
    for lens in ([500, 64], [17, 64], [1, 1], [333, 2]):
        c.cache.lens.copy_(c.ids(lens))
        g.replay()
        c.lens = lens
        c.tokens = [t[:, :, :n] for t, n in zip(c.tokens, lens)] if lens[0] == 500 else c.tokens
        full = c.tokens
        c.tokens = [t[:, :, :n] for t, n in zip(full, lens)]
        c.check((out, lse))
        c.tokens = full
    del g


def test_bad_numbers_are_not_followed(ex):
    """Sequence numbers and table entries out of range: reported, not read; rows of good sequences are right
    (to rounding: where a sequence's sums are cut depends on the whole batch)."""
    c = Case([70, 90, 40], [1, 1, 1], dim=64, page=16, seed=16)
    good = c.cache.table.clone()
    seqs, counts = list(c.seqs), list(c.counts)

    def check(got, rows):
        assert c.cache.status() == ex.EXL3_ERR_INDEX
        for r in rows:
            c.seqs, c.counts, q = [seqs[r]], [1], c.q
            c.q = q[r:r + 1]
            c.check([x[r:r + 1] for x in got])
            c.seqs, c.counts, c.q = list(seqs), list(counts), q

    c.seqs = [0, 3, 2]
    got = c.run()
    assert (got[0][1] == 77).all() and (got[1][1] == 77).all()
    check(got, [0, 2])
    for bad in (-5, c.cache.n_pages, 2 ** 31 - 1):
        c.cache.table[1, 2] = bad
        check(c.run(), [0, 2])
        c.cache.table.copy_(good)
    c.cache.lens[0] = 2 ** 30                                # far past the table: taken as a full row of it
    check(c.run(), [1, 2])


def test_a_repeated_sequence_is_answered_twice(ex):
    c = Case([700, 90], [2, 2], m=2, page=64, seed=19)
    c.seqs, c.counts, c.lens = [0, 1, 0], [2, 2, 2], [700, 90]
    c.q = np.concatenate([c.q, c.q[:1] * 0.5])
    c.check(c.run())


def test_refusals(ex):
    import torch
    c = Case([30, 77], [1, 1], dim=64, seed=17)
    q, seqs = torch.from_numpy(c.q).cuda(), c.ids([0, 1])
    a = c.cache.attention
    for call in (lambda: a(0, seqs, q.float()), lambda: a(0, seqs[:1], q), lambda: a(0, seqs, q[..., :32]),
                 lambda: a(0, seqs, q.cpu()), lambda: a(0, seqs.long(), q), lambda: a(0, seqs, q, counts=seqs[:1]),
                 lambda: a(0, seqs, q, out=q[:, :, :3]), lambda: a(0, seqs, q, out=q.repeat(1, 2, 1, 1)),
                 lambda: a(0, seqs, q, lse=torch.empty(2, 1, 6, dtype=torch.float16, device="cuda")),
                 lambda: a(0, seqs, q[0])):
        with pytest.raises(ValueError):
            call()
    for call, status in ((lambda: a(1, seqs, q), ex.EXL3_ERR_INVALID_ARG), (lambda: a(0, seqs, q, window=-1), ex.EXL3_ERR_INVALID_ARG),
                         (lambda: a(0, seqs, q, sinks=-1), ex.EXL3_ERR_INVALID_ARG),
                         (lambda: a(0, seqs, q, out=q[:1].expand(2, -1, -1, -1)), ex.EXL3_ERR_INVALID_ARG),
                         (lambda: a(0, seqs, q, scale=float("nan")), ex.EXL3_ERR_INVALID_ARG),
                         (lambda: a(0, seqs, q[:, :, :5].contiguous()), ex.EXL3_ERR_UNSUPPORTED),
                         (lambda: a(0, seqs, q.repeat(1, 33, 1, 1)), ex.EXL3_ERR_UNSUPPORTED),
                         (lambda: a(0, seqs, q, workspace=torch.zeros(1024, dtype=torch.uint8, device="cuda")),
                          ex.EXL3_ERR_WORKSPACE)):
        with pytest.raises(ex.Exl3Error) as e:
            call()
        assert e.value.status == status


@pytest.mark.parametrize("m,group", [(1, 4), (12, 4)])                  # both kernels
def test_withheld_tiles_time_out_and_report(ex, m, group):
    """Every copy withheld through the workspace's injection word: the waits run out, the call ends and the
    status says so; with the workspace cleared the next call is right."""
    c = Case([3000, 70, 400], [m, m, m], dim=128, page=64, m=m, group=group, seed=18)
    ws = c.cache.attention_workspace(3, m, 2 * group)
    ws[4:8] = 1
    c.run(workspace=ws)
    assert ex.workspace_status(ws) == ex.EXL3_ERR_TIMEOUT
    ws.zero_()
    c.check(c.run(workspace=ws))
    assert ex.workspace_status(ws) == ex.EXL3_OK


def test_launch_counts(ex):
    """One kernel where the table is short, or the parts of a sequence are few; two otherwise."""
    c = Case([70, 90], [1, 1], kv_heads=2, group=4, dim=64)
    assert c.cache.attention_launches(2, 1, 8) == 1 == c.cache.attention_launches(2, 32, 8)
    d = Case([2000], [1], kv_heads=2, group=4, dim=64, page=64)
    assert d.cache.attention_launches(1, 1, 8) == 2 == d.cache.attention_launches(900, 32, 8)
    assert d.cache.attention_launches(1000, 1, 8) == 1
    assert d.cache.attention_launches(0, 1, 8) == d.cache.attention_launches(1, 33, 8) == d.cache.attention_launches(1, 1, 7) == 0


@pytest.mark.parametrize("m,group", [(1, 5), (3, 5), (5, 7), (16, 5), (32, 8)])
def test_joined_by_the_second_kernel(ex, m, group):
    """Few long sequences, cut into many parts: 16 rows and more, one row tile and several."""
    for heads, dim, lens in ((1, 64, [9000]), (2, 128, [5000, 300, 1200])):
        c = Case(lens, [m] + [max(1, m - 1)] * (len(lens) - 1), kv_heads=heads, group=group, dim=dim, page=64, m=m, seed=m + dim)
        assert c.cache.attention_launches(len(lens), m, heads * group) == 2
        c.check(c.run())


def test_two_streams_with_their_own_workspaces(ex):
    """Two calls on one cache at once: reads only, each with its workspace."""
    import torch
    c = Case([5000, 900], [1, 1], dim=128, page=64, group=4, seed=19)
    q, seqs = torch.from_numpy(c.q).cuda(), c.ids(c.seqs)
    want = c.cache.attention(0, seqs, q)
    streams = [torch.cuda.Stream() for _ in range(3)]
    spaces = [c.cache.attention_workspace(2, 1, 8) for _ in streams]
    outs = [torch.empty_like(want) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, ws, o in zip(streams, spaces, outs):
            c.cache.attention(0, seqs, q, out=o, workspace=ws, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
