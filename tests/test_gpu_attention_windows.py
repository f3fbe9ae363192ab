"""Windows and sinks in the forms that a served model has them: 128 columns,
several row tiles, long sequences cut over CTAs and joined by either kernel,
tables as wide as a model's context."""
import numpy as np
import pytest

from test_gpu_attention import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    from gemm_exl3_gemv_b200 import exl3
    return exl3


def widen(c, tokens):
    """The same cache with a table row for `tokens` tokens."""
    import torch
    from gemm_exl3_gemv_b200.kvcache import KvCache
    old = c.cache
    table = torch.full((old.n_seqs, tokens // c.page), -1, dtype=torch.int32, device="cuda")
    table[:, :old.max_pages] = old.table
    c.cache = KvCache(old.k, old.v, table, old.lens, old.refs, old.free)
    return c


# 5 and 15 rows; 80 rows; two tiles of 128 rows; three of 87, whose borders lie inside a token's heads
ROWS = [(1, 5), (3, 5), (16, 5), (32, 8), (29, 9)]


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("m,group", ROWS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (64, 3), (65, 130), (300, 4), (1000, 70), (4096, 4)])
def test_long_sequences_joined_by_the_second_kernel(ex, window, sinks, m, group, dim):
    """Windows that begin inside a tile and lie differently for the row tiles, sinks that end inside one and that
    meet the window; a sequence shorter than the window, one of the new tokens alone."""
    lens = [5003, 1170, 300, m]
    c = Case(lens, [m, max(1, m - 2), m, m], kv_heads=1, group=group, dim=dim, page=128 if dim == 128 else 16, m=m,
             seed=window % 89 + m)
    assert c.cache.attention_launches(4, m, group) == 2
    c.check(c.run(window=window, sinks=sinks), window=window, sinks=sinks)


@pytest.mark.parametrize("window,sinks", [(0, 0), (200, 5)])
@pytest.mark.parametrize("m,group", ROWS)
def test_short_sequences_in_a_wide_table(ex, m, group, window, sinks):
    """Rows of the table for 131072 tokens, sequences of 1 to 500: the same answers to rounding as from rows that just fit."""
    lens = [m, m + 1, 100 + m, 400 + m]
    c = Case(lens, [m, 1, m, max(1, m - 1)], kv_heads=2, group=group, dim=128, page=64, m=m, seed=m)
    c.check(c.run(window=window, sinks=sinks), window=window, sinks=sinks)
    widen(c, 131072)
    c.check(c.run(window=window, sinks=sinks), window=window, sinks=sinks)


@pytest.mark.parametrize("m,group", [(2, 8), (16, 5), (32, 8)])
def test_unseen_values_of_long_sequences(ex, m, group):
    """Values and keys that are not finite, all along the part between the sinks and the window, and in the
    tokens behind a row's own: no row that does not see them has anything of them."""
    import torch
    window, sinks, n = 700, 5, 4000
    c = Case([n], [m], kv_heads=1, group=group, dim=128, page=64, m=m, seed=m)
    first = n - m - window + 1                               # of the first row's window
    kv = torch.from_numpy(np.stack([x[0, :, 0] for x in c.tokens[0]])).cuda()       # keys, values: (tokens, dim)
    kv[:, sinks:first] = float("nan")
    kv[1, n - 1] = float("inf")                              # the last token's value: seen by the last row alone
    pages = c.cache.table[0, :-(-n // 64)].long()
    for pool, new in ((c.cache.k, kv[0]), (c.cache.v, kv[1])):
        rows = torch.full((len(pages) * 64, 128), float("nan"), dtype=torch.float16, device="cuda")
        rows[:n] = new
        pool[0, pages, 0] = rows.view(-1, 64, 128)
    out, lse = c.run(window=window, sinks=sinks)
    assert torch.isinf(out[0, m - 1]).all() and torch.isfinite(lse).all()
    c.tokens[0][1][0, n - 1] = 0                             # for the rows in front it does not exist
    if m > 1:
        c.counts, c.lens, c.q = [m - 1], [n - 1], c.q[:, :m - 1]
        c.tokens[0] = c.tokens[0][:, :, :n - 1]
        c.m = m - 1
        c.check((out[:, :m - 1], lse[:, :m - 1]), window=window, sinks=sinks)
