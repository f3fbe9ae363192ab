"""Host-side checks of the cache, attention and 4-bit calls (no GPU): argument
validation through the C ABI.  Only invalid calls are made."""
import ctypes

import pytest

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def ex():
    from gemm_exl3_gemv_b200 import build
    build.build()
    from gemm_exl3_gemv_b200 import exl3
    return exl3


def cache(ex, **change):
    d = dict(k=256, v=256, table=256, lens=256, refs=256, free=256, scratch=256, n_layers=2, n_pages=64, n_heads=4,
             page_size=32, head_dim=128, n_seqs=8, max_pages=16)
    d.update(change)
    return ctypes.byref(ex.Cache(**d))


BAD_CACHES = [(dict(k=None), "INVALID_ARG"), (dict(scratch=None), "INVALID_ARG"), (dict(n_layers=0), "INVALID_ARG"),
              (dict(n_pages=-1), "INVALID_ARG"), (dict(max_pages=0), "INVALID_ARG"), (dict(head_dim=80), "UNSUPPORTED"),
              (dict(page_size=48), "UNSUPPORTED"), (dict(page_size=512), "UNSUPPORTED"), (dict(n_heads=257), "UNSUPPORTED"),
              (dict(n_pages=(1 << 20) + 1), "UNSUPPORTED"), (dict(n_seqs=65537), "UNSUPPORTED"),
              (dict(n_layers=1025), "UNSUPPORTED"), (dict(max_pages=1 << 20, page_size=256, n_pages=4), "OK30"),
              (dict(max_pages=(1 << 20) + 1), "UNSUPPORTED"), (dict(n_pages=1 << 20, n_heads=64), "UNSUPPORTED"),
              (dict(v=264), "MISALIGNED"), (dict(table=260), "MISALIGNED")]


@pytest.mark.parametrize("change,status", BAD_CACHES)
def test_bad_caches_are_refused_by_every_call(ex, change, status):
    lib = ex.lib
    c = cache(ex, **change)
    if status == "OK30":                               # 2^28 tokens a sequence: within the limit, refused for the list
        assert lib.exl3_kv_extend(c, 1, 1, None, None, None) == ex.EXL3_ERR_INVALID_ARG
        return
    want = getattr(ex, "EXL3_ERR_" + status)
    assert lib.exl3_kv_reset(c, None) == want
    assert lib.exl3_kv_status(c, None) == want
    assert lib.exl3_kv_compact(c, None) == want
    assert lib.exl3_kv_extend(c, 1, 1, P(16), None, None) == want
    assert lib.exl3_kv_truncate(c, 1, P(16), None, None) == want
    assert lib.exl3_kv_fork(c, 1, P(16), P(16), None) == want
    assert lib.exl3_kv_write(c, 0, 1, 1, P(16), None, P(16), P(16), 0, 0, None) == want
    assert lib.exl3_paged_attention(c, 0, 1, 1, P(16), None, P(16), 0, 0, 8, 1.0, 0, 0, P(16), 0, 0, None, P(256),
                                    1 << 30, None) == want


def test_lists(ex):
    lib, inv, uns, mis = ex.lib, ex.EXL3_ERR_INVALID_ARG, ex.EXL3_ERR_UNSUPPORTED, ex.EXL3_ERR_MISALIGNED
    c = cache(ex)
    for n, p, want in ((0, 16, inv), (-3, 16, inv), (1, 0, inv), (1025, 16, uns), (2, 18, mis)):
        assert lib.exl3_kv_extend(c, n, 1, P(p), None, None) == want
        assert lib.exl3_kv_truncate(c, n, P(p), None, None) == want
        assert lib.exl3_kv_fork(c, n, P(p), P(16), None) == want
        assert lib.exl3_kv_write(c, 0, n, 1, P(p), None, P(16), P(16), 0, 0, None) == want
    assert lib.exl3_kv_fork(c, 1, P(16), P(0), None) == inv
    assert lib.exl3_kv_fork(c, 1, P(16), P(17), None) == mis
    assert lib.exl3_kv_extend(c, 1, 0, P(16), None, None) == inv
    assert lib.exl3_kv_extend(c, 1, 4, P(16), P(6), None) == mis
    assert lib.exl3_kv_truncate(c, 1, P(16), P(5), None) == mis
    assert lib.exl3_kv_extend(None, 1, 1, P(16), None, None) == inv


def test_write(ex):
    f, c = ex.lib.exl3_kv_write, cache(ex)
    call = lambda layer=0, m=1, k=16, v=16, bs=0, rs=0: f(c, layer, 1, m, P(16), None, P(k), P(v), bs, rs, None)
    for kw in (dict(layer=-1), dict(layer=2), dict(m=0), dict(k=0), dict(v=0), dict(bs=-8), dict(rs=-8)):
        assert call(**kw) == ex.EXL3_ERR_INVALID_ARG, kw
    for kw in (dict(k=24), dict(v=24), dict(bs=4), dict(rs=12)):
        assert call(**kw) == ex.EXL3_ERR_MISALIGNED, kw


def test_attention(ex):
    f, c = ex.lib.exl3_paged_attention, cache(ex)
    ok = dict(layer=0, n=1, m=2, seqs=16, counts=0, q=16, qb=0, qr=0, heads=8, scale=1.0, window=0, sinks=0, out=16, ob=0,
              orow=1024, lse=0, ws=256, room=1 << 30)

    def call(**kw):
        a = {**ok, **kw}
        return f(c, a["layer"], a["n"], a["m"], P(a["seqs"]), P(a["counts"]), P(a["q"]), a["qb"], a["qr"], a["heads"],
                 a["scale"], a["window"], a["sinks"], P(a["out"]), a["ob"], a["orow"], P(a["lse"]), P(a["ws"]), a["room"], None)

    need = ex.lib.exl3_paged_attention_workspace_bytes(2, 8, 4, 128)
    assert need > 0
    for kw in (dict(q=0), dict(out=0), dict(m=0), dict(heads=0), dict(layer=2), dict(layer=-1), dict(window=-1), dict(sinks=-1),
               dict(qb=-8), dict(orow=-8), dict(scale=float("inf")), dict(scale=float("nan")), dict(n=0), dict(seqs=0)):
        assert call(**kw) == ex.EXL3_ERR_INVALID_ARG, kw
    for kw in (dict(m=33), dict(heads=6), dict(heads=132), dict(n=1025)):
        assert call(**kw) == ex.EXL3_ERR_UNSUPPORTED, kw
    for kw in (dict(q=24), dict(out=24), dict(lse=20), dict(qb=4), dict(qr=4), dict(ob=4), dict(orow=1028), dict(ws=16), dict(counts=3)):
        assert call(**kw) == ex.EXL3_ERR_MISALIGNED, kw
    for kw in (dict(ws=0), dict(room=need - 1)):
        assert call(**kw) == ex.EXL3_ERR_WORKSPACE, kw
    # rows of the result (1024 elements each) must lie apart
    for kw in (dict(orow=0), dict(orow=1016), dict(n=2, ob=1024), dict(n=2, ob=2040), dict(n=2, ob=0), dict(n=2, m=1, ob=1016),
               dict(n=3, ob=1024, orow=2048), dict(n=3, ob=1024, orow=3064)):
        assert call(**kw) == ex.EXL3_ERR_INVALID_ARG, kw
    for kw in (dict(m=1, orow=0), dict(n=2, ob=2048), dict(n=2, m=1, ob=1024, orow=0), dict(n=3, ob=1024, orow=3 * 1024)):
        assert call(**kw, ws=0) == ex.EXL3_ERR_WORKSPACE, kw      # refused for the workspace alone


def test_sizes(ex):
    w = ex.lib.exl3_paged_attention_workspace_bytes
    for bad in ((0, 8, 4, 128), (33, 8, 4, 128), (1, 8, 0, 128), (1, 0, 4, 128), (1, 6, 4, 128), (1, 132, 4, 128), (1, 8, 4, 96)):
        assert w(*bad) == 0, bad
    assert w(32, 40, 8, 128) >= w(1, 40, 8, 128) > w(1, 40, 8, 64) > 0
    s = ex.lib.exl3_kv_scratch_bytes
    assert s(0) == s(-1) == s((1 << 20) + 1) == 0
    assert s(1 << 20) >= 4 << 20 and s(1) > 0
    q = ex.q4_workspace_bytes
    for bad in ((0, 64, 16), (33, 64, 16), (1, 96, 16), (1, 64, 24), (1, 0, 16), (1, 64, -16), (1, (1 << 20) + 64, 16),
                (1, 64, (1 << 20) + 16)):
        assert q(*bad) == 0, bad
    assert q(1, 64, 16) > 0 and q(32, 17408, 5120) > 0
    for shape in ((1024, 4096), (17408, 1024), (2048, 2048), (64, 16), (5120, 33024)):
        sizes = [q(m, *shape) for m in range(1, 33)]
        assert sizes == sorted(sizes)                   # enough for fewer rows too


def test_q4(ex):
    f = ex.lib.exl3_q4_gemm
    ok = dict(m=1, x=16, packed=16, scale=16, zero=0, y=16, k=256, n=64, group=64, ws=256, room=1 << 24)

    def call(**kw):
        a = {**ok, **kw}
        return f(a["m"], P(a["x"]), P(a["packed"]), P(a["scale"]), P(a["zero"]), P(a["y"]), 0, a["k"], a["n"], a["group"],
                 P(a["ws"]), a["room"], None)

    for kw in (dict(m=0), dict(x=0), dict(packed=0), dict(scale=0), dict(y=0), dict(k=0), dict(n=-16)):
        assert call(**kw) == ex.EXL3_ERR_INVALID_ARG, kw
    for kw in (dict(m=33), dict(k=96), dict(n=24), dict(group=16), dict(group=256), dict(k=64, group=128), dict(k=192, group=128)):
        assert call(**kw) == ex.EXL3_ERR_UNSUPPORTED, kw
    for kw in (dict(x=18), dict(packed=20), dict(scale=18), dict(zero=17), dict(y=20), dict(ws=16)):
        assert call(**kw) == ex.EXL3_ERR_MISALIGNED, kw
    for kw in (dict(ws=0), dict(room=255)):
        assert call(**kw) == ex.EXL3_ERR_WORKSPACE, kw
    g = ex.lib.exl3_q4_pack
    assert g(P(0), 64, 16, P(16), None) == ex.EXL3_ERR_INVALID_ARG
    assert g(P(16), 64, 0, P(16), None) == ex.EXL3_ERR_INVALID_ARG
    assert g(P(16), 96, 16, P(16), None) == ex.EXL3_ERR_UNSUPPORTED
    assert g(P(16), 64, 16, P(24), None) == ex.EXL3_ERR_MISALIGNED


def test_attention_launches(ex):
    f = ex.lib.exl3_paged_attention_launches
    c = cache(ex)                                       # 16 pages of 32: eight tiles of 64 tokens
    assert f(c, 1, 1, 8) == f(c, 1, 32, 8) == 1
    c = cache(ex, max_pages=4096)
    assert f(c, 1, 1, 8) == f(c, 1, 32, 8) == f(c, 500, 32, 8) == 2 and f(c, 500, 1, 8) == 1
    assert f(c, 0, 1, 8) == f(c, 1025, 1, 8) == f(c, 1, 0, 8) == f(c, 1, 33, 8) == f(c, 1, 1, 6) == f(cache(ex, k=None), 1, 1, 8) == 0


def test_compiled_binding(ex):
    """The compiled calls hand over every argument as ctypes does: the same status whichever argument is wrong.
    Every call is refused for its last check (no room, a misaligned list or stride) if for nothing before it."""
    b, desc = ex._binding, cache(ex)._obj
    at = ctypes.addressof(desc)
    inv, uns, mis = ex.EXL3_ERR_INVALID_ARG, ex.EXL3_ERR_UNSUPPORTED, ex.EXL3_ERR_MISALIGNED
    wrong = {                                            # the call; argument: values and what they give
        "exl3_q4_gemm": ([1, 16, 16, 16, 16, 16, 0, 256, 64, 64, 256, 0, 0],
                         {0: [(0, inv), (33, uns)], 1: [(None, inv), (18, mis)], 2: [(None, inv), (18, mis)],
                          3: [(None, inv), (18, mis)], 4: [(17, mis)], 5: [(None, inv), (18, mis)], 7: [(0, inv), (96, uns)],
                          8: [(0, inv), (24, uns)], 9: [(48, uns)]}),
        "exl3_kv_extend": ([at, 1, 1, 17, 16, 0], {0: [(None, inv)], 1: [(0, inv), (1025, uns)], 2: [(0, inv)], 3: [(None, inv)]}),
        "exl3_kv_write": ([at, 0, 1, 1, 16, 16, 16, 16, 4, 4, 0],
                          {0: [(None, inv)], 1: [(-1, inv), (2, inv)], 2: [(0, inv), (1025, uns)], 3: [(0, inv)], 4: [(None, inv)],
                           6: [(None, inv)], 7: [(None, inv)], 8: [(-8, inv)], 9: [(-8, inv)]}),
        "exl3_kv_truncate": ([at, 1, 17, 16, 0], {0: [(None, inv)], 1: [(0, inv), (1025, uns)], 2: [(None, inv)]}),
        "exl3_kv_fork": ([at, 1, 16, 17, 0], {0: [(None, inv)], 1: [(0, inv), (1025, uns)], 2: [(None, inv)], 3: [(None, inv)]}),
        "exl3_kv_compact": ([None, 0], {}),
        "exl3_paged_attention": ([at, 0, 1, 2, 16, 16, 16, 64, 64, 8, 1.0, 0, 0, 16, 1024, 1024, 16, 256, 0, 0],
                                 {0: [(None, inv)], 1: [(2, inv)], 2: [(0, inv), (1025, uns)], 3: [(0, inv), (33, uns)], 4: [(None, inv)],
                                  5: [(3, mis)], 6: [(None, inv), (24, mis)], 7: [(-8, inv), (4, mis)], 8: [(-8, inv), (4, mis)],
                                  9: [(0, inv), (6, uns)], 10: [(float("inf"), inv)], 11: [(-1, inv)], 12: [(-1, inv)],
                                  13: [(None, inv), (24, mis)], 14: [(-8, inv), (4, mis)], 15: [(-8, inv), (1016, inv), (1028, mis)],
                                  16: [(20, mis)]}),
    }
    assert set(wrong) == set(b.NAMES)
    for name, (args, changes) in wrong.items():
        call, reference = getattr(b, name[len("exl3_"):]), getattr(ex.lib, name)
        base = call(*args)
        assert base == reference(*args) != ex.EXL3_OK
        for i, values in changes.items():
            for value, status in values:
                one = args[:i] + [value] + args[i + 1:]
                assert call(*one) == reference(*one) == status, (name, i, value)
        with pytest.raises(TypeError):
            call(*args[:-1])
        with pytest.raises(TypeError):
            call(*args[:-1], "0")
    with pytest.raises(OverflowError):
        b.kv_extend(at, 1 << 40, 1, 17, None, 0)


def test_status_strings(ex):
    assert b"CACHE_FULL" in ex.lib.exl3_status_string(ex.EXL3_ERR_CACHE_FULL)
    assert b"INDEX" in ex.lib.exl3_status_string(ex.EXL3_ERR_INDEX)


def test_tensor_checks_without_a_gpu(ex):
    """The binding refuses tensors of the wrong place before it calls the library."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("where there is a GPU the GPU tests cover it")
    x = torch.zeros(1, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        ex.q4_gemm(x, torch.zeros(1, 1, 32, 4, dtype=torch.int32), torch.zeros(1, 16, dtype=torch.float16), group=64)
    from gemm_exl3_gemv_b200.kvcache import KvCache
    kv = torch.zeros(1, 4, 1, 16, 64, dtype=torch.float16)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    with pytest.raises(ValueError):
        KvCache(kv, kv, i(2, 2), i(2), i(4), i(1))
