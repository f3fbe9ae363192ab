"""Cases of the cache, attention and 4-bit product operators, for measuring them.

``run`` makes one pass through an operator: with ``own`` the library's calls, otherwise the same thing in
elementary torch operations in 32 bits.  ``exact`` evaluates the definitions in 64 bits.

Kinds of cases:
  q4      y = x W for 4-bit weights with group scales and zero points, 1 to 32 rows
  attn    attention of the last m tokens of each sequence over a paged cache (window 0: all tokens visible)
  append  sequences grow by new tokens, whose keys and values are written in every layer
  pages   finished sequences leave, others are forked, the pool is compacted
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # a small adapter or draft-model matrix for a handful of drafted tokens, odd row count: latency counts
        dict(name="q4 m7 256x384", kind="q4", m=7, k=256, n=384, group=32, fp32=True),
        # decode through the attention output projection of a 27B-class layer
        dict(name="q4 m1 5120x5120", kind="q4", m=1, k=5120, n=5120, group=128, fp32=False),
        # verification of 32 drafted rows through an MLP gate of that layer
        dict(name="q4 m32 5120x17408", kind="q4", m=32, k=5120, n=17408, group=128, fp32=False),
        # first tokens of one short chat: the smallest attention call
        dict(name="attn decode 1x100", kind="attn", batch=1, length=100, m=1, kv_heads=8, group=5, dim=128, page=64,
             window=0, sinks=0, layers=1),
        # ordinary decode of a batch of ragged chats
        dict(name="attn decode 32x4000", kind="attn", batch=32, length=4000, m=1, kv_heads=8, group=5, dim=128,
             page=64, window=0, sinks=0, layers=1),
        # decode of one long document: work is split over the length
        dict(name="attn decode 1x131077", kind="attn", batch=1, length=131077, m=1, kv_heads=8, group=5, dim=128,
             page=64, window=0, sinks=0, layers=1),
        # decode of ragged sequences under a sliding window with sinks, small pages and heads
        dict(name="attn window 24x9001", kind="attn", batch=24, length=9001, m=1, kv_heads=4, group=8, dim=64,
             page=16, window=1000, sinks=4, layers=1),
        # verification of 16 drafted tokens per sequence under a window
        dict(name="attn window verify 8x16", kind="attn", batch=8, length=8192, m=16, kv_heads=8, group=5, dim=128,
             page=128, window=4096, sinks=4, layers=1),
        # one token for each sequence of a decode batch, two layers of the cache
        dict(name="append 64x1", kind="append", batch=64, length=700, m=1, kv_heads=8, dim=128, page=64, layers=2,
             forked=8),
        # a prompt is taken in
        dict(name="append 2x2001", kind="append", batch=2, length=333, m=2001, kv_heads=8, dim=128, page=64, layers=2,
             forked=0),
        # a few sequences: two leave, two are forked
        dict(name="pages 8 sequences", kind="pages", seqs=8, length=150, gone=2, forks=2, kv_heads=4, dim=64, page=16,
             layers=1),
        # a full pool loses a third of its sequences
        dict(name="pages 48 sequences", kind="pages", seqs=48, length=2500, gone=16, forks=16, kv_heads=8, dim=128,
             page=64, layers=2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["q4", "attn", "attn", "append", "pages"])
    if kind == "q4":
        while True:
            group = rng.choice([32, 64, 128])
            k = max(1, _log(rng, 128, 17408) // max(group, 64)) * max(group, 64)
            n = max(1, _log(rng, 16, 17408) // 16) * 16
            if k * n <= 5120 * 17408:
                return dict(kind=kind, m=_log(rng, 1, 32), k=k, n=n, group=group, fp32=rng.random() < 0.5)
    dim = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128, 256])
    if kind == "attn":
        length = _log(rng, 1, 131072)
        batch = max(1, min(_log(rng, 1, 64), 131072 // length))
        m = min(length, 1 if rng.random() < 0.5 else _log(rng, 2, 32))
        windowed = rng.random() < 0.4
        kv_heads, group = rng.choice([1, 2, 4, 8]), rng.randint(1, 8)
        while m > 1 and batch * length * m * group * kv_heads > 8 * 8192 * 16 * 40:
            m = m // 2
        return dict(kind=kind, batch=batch, length=length, m=m, kv_heads=kv_heads, group=group, dim=dim, page=page,
                    window=_log(rng, 1, 8192) if windowed else 0, sinks=rng.randint(0, 70) if windowed else 0, layers=1)
    kv_heads, layers = rng.choice([1, 2, 4, 8]), rng.randint(1, 2)
    if kind == "append":
        m = _log(rng, 1, 2000)
        batch = max(1, min(_log(rng, 1, 100), 4000 // m))
        return dict(kind=kind, batch=batch, length=_log(rng, 1, 900), m=m, kv_heads=kv_heads, dim=dim, page=page,
                    layers=layers, forked=rng.randint(0, batch // 2))
    seqs = _log(rng, 3, 48)
    return dict(kind=kind, seqs=seqs, length=_log(rng, 20, 2500), gone=rng.randint(1, seqs // 3),
                forks=rng.randint(1, seqs // 3), kv_heads=kv_heads, dim=dim, page=page, layers=layers)


# ----------------------------------------------------------------- inputs ---

def _lengths(count, most, least=1):
    """Ragged lengths, the longest first (the same for every seed: the work of a case does not depend on it)."""
    r = random.Random(77 + count)
    return [max(least, most if i == 0 else int(most * r.uniform(0.2, 1.0))) for i in range(count)]


def _counts(case):
    """New tokens of each sequence: all m, or fewer for some sequences of a batch."""
    r = random.Random(5 + case["batch"])
    return [case["m"] if i % 3 == 0 else r.randint(1, case["m"]) for i in range(case["batch"])]


def _attn_lengths(case):
    return _lengths(case["batch"], case["length"], min(case["length"], case["m"]))


def _order(count):
    """The sequences of a batch, in the batch's order."""
    ids = list(range(count))
    random.Random(3 + count).shuffle(ids)
    return ids


def _up(a, b):
    return -(-a // b)


def _pool(g, lens, n_seqs, n_pages, max_pages, case, fill):
    """Pages and bookkeeping of a cache whose first len(lens) sequences hold lens[i] tokens on scattered pages.

    The bookkeeping is one flat int32 buffer with the views table (-1: no page), lens, refs and free (bit p%32 of
    word p/32 is set while page p is free)."""
    ps, h, d, nl = case["page"], case["kv_heads"], case["dim"], case["layers"]
    shape = (nl, n_pages, h, ps, d)
    k = torch.zeros(shape, dtype=torch.float16, device=DEV)
    v = torch.zeros(shape, dtype=torch.float16, device=DEV)
    if fill:
        k.normal_(generator=g)
        v.normal_(generator=g)
    words = _up(n_pages, 32)
    sizes = [n_seqs * max_pages, n_seqs, n_pages, words]
    starts = [0]
    for s in sizes:
        starts.append(starts[-1] + _up(s, 64) * 64)
    book = torch.zeros(starts[-1], dtype=torch.int32, device=DEV)
    table, lens_t, refs, free = (book[a:a + s] for a, s in zip(starts, sizes))
    table = table.view(n_seqs, max_pages)
    need = [_up(n, ps) for n in lens]
    order = torch.randperm(n_pages, generator=g, device=DEV)[:sum(need)].to(torch.int32)
    rows = torch.full((n_seqs, max_pages), -1, dtype=torch.int32, device=DEV)
    at = 0
    for i, c in enumerate(need):
        rows[i, :c] = order[at:at + c]
        at += c
    table.copy_(rows)
    lens_t[:len(lens)] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    refs[order.long()] = 1
    free.copy_(_bits(refs == 0))
    return dict(k=k, v=v, book=book, table=table, lens=lens_t, refs=refs, free=free)


def _share(st, src, dst, ps):
    """Sequence dst takes all pages of src as well (a fork, made while the inputs are prepared)."""
    n = _up(int(st["lens"][src]), ps)
    st["table"][dst] = st["table"][src]
    st["lens"][dst] = st["lens"][src]
    st["refs"][st["table"][src, :n].long()] += 1


def _ids(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    kind = case["kind"]
    st = {"case": case}
    rand = lambda *s: torch.randn(s, generator=g, device=DEV)
    if kind == "q4":
        m, k, n, gr = case["m"], case["k"], case["n"], case["group"]
        st["x"] = rand(m, k).half()
        st["packed"] = torch.randint(-2 ** 31, 2 ** 31, (n // 16, k // 64, 32, 4), generator=g, device=DEV,
                                     dtype=torch.int64).to(torch.int32)
        st["scale"] = ((0.5 + torch.rand((k // gr, n), generator=g, device=DEV)) * 0.2 / math.sqrt(k)).half()
        st["zero"] = torch.randint(0, 16, (k // gr, n), generator=g, device=DEV).to(torch.uint8)
        if own:
            from gemm_exl3_gemv_b200 import exl3
            st["ws"] = exl3.q4_alloc_workspace(m, k, n)
        return st
    ps = case["page"]
    if kind == "attn":
        lens = _attn_lengths(case)
        need = sum(_up(n, ps) for n in lens)
        st.update(_pool(g, lens, case["batch"], need + 3, _up(case["length"], ps), case, True))
        b, m, hq, d = case["batch"], case["m"], case["kv_heads"] * case["group"], case["dim"]
        st["q"] = (1.5 * rand(b, m, hq, d)).half()
        st["counts"] = _ids(_counts(case))
        st["seqs"] = _ids(_order(b))
        st["out"] = torch.zeros((b, m, hq, d), dtype=torch.float16, device=DEV)
        st["lse"] = torch.zeros((b, m, hq), dtype=torch.float32, device=DEV)
    elif kind == "append":
        b, m = case["batch"], case["m"]
        lens = _lengths(b, case["length"])
        longest = _up(case["length"] + m, ps)
        n_pages = sum(_up(n, ps) + _up(m, ps) + 2 for n in lens)
        st.update(_pool(g, lens, b + 1, n_pages, longest, case, True))
        for i in range(case["forked"]):          # pairs of sequences that share every page
            src, dst = 2 * i, 2 * i + 1
            old = _up(lens[dst], ps)
            st["refs"][st["table"][dst, :old].long()] -= 1
            _share(st, src, dst, ps)
        st["free"].copy_(_bits(st["refs"] == 0))
        st["seqs"] = torch.arange(b, dtype=torch.int32, device=DEV)
        st["counts"] = _ids(_counts(case))
        st["k_new"] = rand(case["layers"], b, m, case["kv_heads"], case["dim"]).half()
        st["v_new"] = rand(case["layers"], b, m, case["kv_heads"], case["dim"]).half()
        st["book0"] = st["book"].clone()
    else:
        n = case["seqs"]
        lens = _lengths(n, case["length"])
        need = sum(_up(x, ps) for x in lens)
        st.update(_pool(g, lens, n + case["forks"], need + 2, _up(case["length"], ps), case, True))
        order = torch.randperm(n, generator=g, device=DEV).to(torch.int32)
        st["gone"] = order[:case["gone"]].contiguous()
        st["src"] = order[case["gone"]:case["gone"] + case["forks"]].contiguous()
        st["dst"] = torch.arange(n, n + case["forks"], dtype=torch.int32, device=DEV)
        st["book0"] = st["book"].clone()
    if own:
        from gemm_exl3_gemv_b200.kvcache import KvCache
        st["cache"] = KvCache(st["k"], st["v"], st["table"], st["lens"], st["refs"], st["free"])
        if kind == "attn":
            st["ws"] = st["cache"].attention_workspace(case["batch"], case["m"], st["q"].shape[2])
    return st


# ------------------------------------------------------------ plain forms ---

def _bits(flags):
    """Truth values as bits of int32 words."""
    n = flags.numel()
    pad = torch.zeros(_up(n, 32) * 32, dtype=torch.int64, device=flags.device)
    pad[:n] = flags
    w = (pad.view(-1, 32) << torch.arange(32, device=flags.device)).sum(1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


def _q4_weights(packed, scale, zero, group):
    """The (k, n) matrix in 32 bits.  Word j of lane 4 g + t of tile (tn, tk) holds channels 16 tn + g + 8 c and
    inputs 64 tk + 32 (j / 2) + 8 t + 4 (j % 2) + i, i = 0..3, at bits 4 c + 8 (i / 2) + 16 (i % 2)."""
    tn, tk = packed.shape[:2]
    w = packed.view(tn, tk, 8, 4, 2, 2, 1, 1)
    c = torch.arange(2, device=w.device, dtype=torch.int32).view(2, 1)
    i = torch.arange(4, device=w.device, dtype=torch.int32)
    q = (w >> (4 * c + 8 * (i // 2) + 16 * (i % 2))) & 15          # tn, tk, g, t, j / 2, j % 2, c, i
    q = q.permute(1, 4, 3, 5, 7, 0, 6, 2).reshape(64 * tk, 16 * tn).float()
    z = zero.float().repeat_interleave(group, 0)
    return (q - z) * scale.float().repeat_interleave(group, 0)


def _visible(pos, tokens, window, sinks):
    """Which tokens the query at each position sees: pos (...,), tokens (T,) -> (..., T)."""
    pos = pos.unsqueeze(-1)
    see = tokens <= pos
    if window:
        see = see & ((tokens > pos - window) | (tokens < sinks))
    return see


def _plain_attention(st):
    case = st["case"]
    b, m, hk, gr, d, ps = (case[x] for x in ("batch", "m", "kv_heads", "group", "dim", "page"))
    seqs = st["seqs"].long()
    lens, counts = st["lens"][seqs], st["counts"]
    pages = st["table"][seqs].clamp(min=0).long()
    t = pages.shape[1] * ps
    k = st["k"][0][pages].permute(0, 2, 1, 3, 4).reshape(b, hk, t, d).float()
    v = st["v"][0][pages].permute(0, 2, 1, 3, 4).reshape(b, hk, t, d).float()
    row = torch.arange(m, device=DEV)
    pos = (lens - counts).unsqueeze(1) + row                                      # b, m
    see = _visible(pos, torch.arange(t, device=DEV), case["window"], case["sinks"])
    q = st["q"].float().view(b, m, hk, gr, d).permute(0, 2, 1, 3, 4).reshape(b, hk, m * gr, d)
    s = (q @ k.transpose(2, 3)).view(b, hk, m, gr, t) * (1.0 / math.sqrt(d))
    s = s.masked_fill(~see.view(b, 1, m, 1, t), float("-inf"))
    top = s.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = (s - top).exp()
    total = p.sum(-1, keepdim=True)
    o = (p.view(b, hk, m * gr, t) @ v).view(b, hk, m, gr, d) / total.clamp(min=1e-37)
    lse = top + total.log()
    mine = (row < counts.unsqueeze(1)).view(b, m, 1)
    o = o.permute(0, 2, 1, 3, 4).reshape(b, m, hk * gr, d)
    lse = lse.permute(0, 2, 1, 3, 4).reshape(b, m, hk * gr)
    st["out"].copy_(torch.where(mine.unsqueeze(-1), o.half(), st["out"]))
    st["lse"].copy_(torch.where(mine, lse, st["lse"]))
    return {"out": st["out"], "lse": st["lse"]}


def _plain_truncate(st, seqs, new_lens, ps):
    """The listed sequences keep their first new_lens tokens; pages that nobody holds any more are free."""
    rows, old = st["table"][seqs], st["lens"][seqs]
    new = torch.minimum(old, new_lens)
    at = torch.arange(rows.shape[1], device=DEV)
    drop = (at >= ((new + ps - 1) // ps).unsqueeze(1)) & (at < ((old + ps - 1) // ps).unsqueeze(1))
    st["refs"].index_put_((rows[drop].long(),), torch.tensor(-1, dtype=torch.int32, device=DEV), accumulate=True)
    st["table"][seqs] = torch.where(drop, torch.full_like(rows, -1), rows)
    st["lens"][seqs] = new
    st["free"].copy_(_bits(st["refs"] == 0))


def _plain_extend(st, seqs, counts, ps):
    """Pages for the new tokens: lowest free page first, in batch order; a partly filled shared page is replaced by
    a copy of its tokens."""
    rows, old = st["table"][seqs], st["lens"][seqs]
    at = torch.arange(rows.shape[1], device=DEV)
    last = rows.gather(1, (old // ps).clamp(max=rows.shape[1] - 1).long().unsqueeze(1)).squeeze(1)
    shared = (old % ps != 0) & (counts > 0) & (st["refs"][last.clamp(min=0).long()] > 1)
    new = old + counts
    fresh = (at >= ((old + ps - 1) // ps).unsqueeze(1)) & (at < ((new + ps - 1) // ps).unsqueeze(1))
    fresh = fresh | (shared.unsqueeze(1) & (at == (old // ps).unsqueeze(1)))
    pages = (st["refs"] == 0).nonzero().squeeze(1)[:int(fresh.sum())]
    got = torch.full_like(rows, -1)
    got[fresh] = pages.to(torch.int32)
    st["table"][seqs] = torch.where(fresh, got, rows)
    to = got.gather(1, (old // ps).clamp(max=rows.shape[1] - 1).long().unsqueeze(1)).squeeze(1)[shared].long()
    come = last[shared].long()
    keep = (torch.arange(ps, device=DEV) < (old[shared] % ps).unsqueeze(1)).view(1, -1, 1, ps, 1)
    st["k"][:, to] = torch.where(keep, st["k"][:, come], st["k"][:, to])
    st["v"][:, to] = torch.where(keep, st["v"][:, come], st["v"][:, to])
    one = torch.tensor(1, dtype=torch.int32, device=DEV)
    st["refs"].index_put_((pages,), one, accumulate=True)
    st["refs"].index_put_((come,), -one, accumulate=True)
    st["lens"][seqs] = new
    st["free"].copy_(_bits(st["refs"] == 0))


def _plain_write(st, seqs, counts, ps):
    """Every layer's new keys and values at the last counts places of each sequence."""
    m = st["k_new"].shape[2]
    row = torch.arange(m, device=DEV)
    pos = (st["lens"][seqs] - counts).unsqueeze(1) + row
    mine = row < counts.unsqueeze(1)
    page = st["table"][seqs].gather(1, (pos // ps).clamp(max=st["table"].shape[1] - 1).long())[mine].long()
    slot = (pos % ps)[mine].long()
    st["k"][:, page, :, slot] = st["k_new"][:, mine].transpose(0, 1)
    st["v"][:, page, :, slot] = st["v_new"][:, mine].transpose(0, 1)


def _plain_fork(st, src, dst, ps):
    rows, n = st["table"][src], st["lens"][src]
    at = torch.arange(rows.shape[1], device=DEV)
    held = at < ((n + ps - 1) // ps).unsqueeze(1)
    st["refs"].index_put_((rows[held].long(),), torch.tensor(1, dtype=torch.int32, device=DEV), accumulate=True)
    st["table"][dst] = torch.where(held, rows, torch.full_like(rows, -1))
    st["lens"][dst] = n


def _plain_compact(st):
    """Used pages end up in front: the i-th used page behind the border takes the i-th free place before it."""
    used = st["refs"] > 0
    n = int(used.sum())
    come = used[n:].nonzero().squeeze(1) + n
    to = (~used[:n]).nonzero().squeeze(1)
    st["k"][:, to] = st["k"][:, come]
    st["v"][:, to] = st["v"][:, come]
    names = torch.arange(used.numel(), dtype=torch.int32, device=DEV)
    names[come] = to.to(torch.int32)
    st["table"].copy_(torch.where(st["table"] >= 0, names[st["table"].clamp(min=0).long()], st["table"]))
    st["refs"][to] = st["refs"][come]
    st["refs"][come] = 0
    st["free"].copy_(_bits(st["refs"] == 0))


# -------------------------------------------------------------------- run ---

def _cache(st):
    return {x: st[x] for x in ("table", "lens", "refs", "free", "k", "v")}


def run(st):
    case = st["case"]
    kind = case["kind"]
    if kind == "q4":
        if own:
            from gemm_exl3_gemv_b200 import exl3
            return exl3.q4_gemm(st["x"], st["packed"], st["scale"], st["zero"], case["group"], fp32=case["fp32"],
                                workspace=st["ws"])
        y = st["x"].float() @ _q4_weights(st["packed"], st["scale"], st["zero"], case["group"])
        return y if case["fp32"] else y.half()
    if kind == "attn":
        if own:
            st["cache"].attention(0, st["seqs"], st["q"], counts=st["counts"], window=case["window"],
                                  sinks=case["sinks"], out=st["out"], lse=st["lse"], workspace=st["ws"])
            return {"out": st["out"], "lse": st["lse"]}
        return _plain_attention(st)
    ps = case["page"]
    # the bookkeeping starts every pass as it was, so that each pass moves the same pages
    st["book"].copy_(st["book0"])
    if kind == "append":
        if own:
            c = st["cache"]
            c.extend(st["seqs"], case["m"], counts=st["counts"])
            for layer in range(case["layers"]):
                c.write(layer, st["seqs"], st["k_new"][layer], st["v_new"][layer], counts=st["counts"])
        else:
            _plain_extend(st, st["seqs"].long(), st["counts"], ps)
            _plain_write(st, st["seqs"].long(), st["counts"], ps)
        return _cache(st)
    if own:
        c = st["cache"]
        c.truncate(st["gone"])
        c.fork(st["src"], st["dst"])
        c.compact()
    else:
        _plain_truncate(st, st["gone"].long(), torch.zeros_like(st["gone"]), ps)
        _plain_fork(st, st["src"].long(), st["dst"].long(), ps)
        _plain_compact(st)
    return _cache(st)


# ------------------------------------------------------------------- work ---

def work(case):
    kind = case["kind"]
    if kind == "q4":
        m, k, n, g = case["m"], case["k"], case["n"], case["group"]
        return {"bytes": k * n / 2 + 3 * (k // g) * n + 2 * m * k + (4 if case["fp32"] else 2) * m * n,
                "flops": 2 * m * k * n}
    hk, d, ps = case["kv_heads"], case["dim"], case["page"]
    if kind == "attn":
        hq, w, s = hk * case["group"], case["window"], case["sinks"]
        tokens = pairs = rows = 0
        lens = _attn_lengths(case)
        for i, c in zip(_order(case["batch"]), _counts(case)):
            n = lens[i]
            first = n - c                                  # position of the first new token
            if w:
                tokens += min(n, max(0, n - max(0, first - w + 1)) + min(s, max(0, first - w + 1)))
                pairs += sum(min(p + 1, w + min(s, max(0, p - w + 1))) for p in range(first, n))
            else:
                tokens += n
                pairs += sum(range(first + 1, n + 1))
            rows += c
        return {"bytes": 4 * d * hk * tokens + rows * hq * (4 * d + 4), "flops": 4 * d * hq * pairs}
    token = 4 * hk * d * case["layers"]                     # key and value bytes of one token
    if kind == "append":
        return {"bytes": 2 * token * sum(_counts(case)), "flops": 0}
    # the pages of the sequences that left, on average: those of them that lie before the border are filled again
    need = [_up(n, ps) for n in _lengths(case["seqs"], case["length"])]
    total = sum(need) + 2
    left = total * (1 - case["gone"] / case["seqs"])
    return {"bytes": 2 * token * ps * left * (1 - left / total) + 8 * total, "flops": 0}


# ------------------------------------------------------------------ exact ---

def exact(case, seed):
    st = _inputs(case, seed)
    kind = case["kind"]
    if kind == "q4":
        return _exact_q4(case, st)
    if kind == "attn":
        return _exact_attention(case, st)
    return _exact_append(case, st) if kind == "append" else _exact_pages(case, st)


def _inputs(case, seed):
    global own
    was, own = own, False
    try:
        return prepare(case, seed)
    finally:
        own = was


def _exact_q4(case, st):
    """Weight by weight from the packed words: each of a word's eight 4-bit fields goes to its place."""
    k, n = case["k"], case["n"]
    words = st["packed"].long() & 0xFFFFFFFF
    lane = torch.arange(32, device=DEV)
    w = torch.zeros((k, n), dtype=torch.float64, device=DEV)
    tk, tn = torch.arange(k // 64, device=DEV), torch.arange(n // 16, device=DEV)
    for j in range(4):
        for field in range(8):
            low, c = field % 4, field % 2
            i = 2 * (low // 2) + field // 4
            rows = 64 * tk.view(1, -1, 1) + 32 * (j // 2) + 8 * (lane % 4) + 4 * (j % 2) + i
            cols = 16 * tn.view(-1, 1, 1) + lane // 4 + 8 * c
            w[rows, cols] = ((words[:, :, :, j] >> (4 * field)) % 16).double()
    for a in range(k // case["group"]):
        part = slice(a * case["group"], (a + 1) * case["group"])
        w[part] = st["scale"][a].double() * (w[part] - st["zero"][a].double())
    return torch.mm(st["x"].double(), w)


def _exact_attention(case, st):
    b, m, hk, gr, d, ps = (case[x] for x in ("batch", "m", "kv_heads", "group", "dim", "page"))
    out, lse = st["out"].double(), st["lse"].double()
    for i, (s, c) in enumerate(zip(st["seqs"].tolist(), st["counts"].tolist())):
        n = int(st["lens"][s])
        held = st["table"][s, :_up(n, ps)].tolist()
        k = torch.cat([st["k"][0, p] for p in held], 1)[:, :n].double()            # hk, n, d
        v = torch.cat([st["v"][0, p] for p in held], 1)[:, :n].double()
        for r in range(c):
            p = n - c + r
            see = list(range(p + 1))
            if case["window"]:
                lo = max(0, p + 1 - case["window"])
                see = list(range(min(case["sinks"], lo))) + list(range(lo, p + 1))
            contiguous = len(see) == p + 1
            kk = k[:, :p + 1] if contiguous else k[:, see]
            vv = v[:, :p + 1] if contiguous else v[:, see]
            q = st["q"][i, r].double().view(hk, gr, d)
            a = torch.einsum("hgd,htd->hgt", q, kk) / math.sqrt(d)
            lse[i, r] = torch.logsumexp(a, 2).reshape(-1)
            out[i, r] = torch.einsum("hgt,htd->hgd", torch.softmax(a, 2), vv).reshape(hk * gr, d)
    return {"out": out, "lse": lse}


def _lists(st):
    return st["table"].tolist(), st["lens"].tolist(), st["refs"].tolist()


def _answer(st, table, lens, refs, k, v):
    words = [0] * st["free"].numel()
    for p, r in enumerate(refs):
        if r == 0:
            words[p // 32] |= 1 << (p % 32)
    words = [w - 2 ** 32 if w >= 2 ** 31 else w for w in words]
    return {"table": _ids(table), "lens": _ids(lens), "refs": _ids(refs), "free": _ids(words), "k": k.double(),
            "v": v.double()}


def _exact_append(case, st):
    """Sequence after sequence, page after page."""
    ps, k, v = case["page"], st["k"], st["v"]
    table, lens, refs = _lists(st)
    before = list(refs)
    free = [p for p, r in enumerate(refs) if r == 0]
    for b, (s, c) in enumerate(zip(st["seqs"].tolist(), st["counts"].tolist())):
        n = lens[s]
        if c and n % ps and before[table[s][n // ps]] > 1:
            old, new = table[s][n // ps], free.pop(0)
            for a in (k, v):
                a[:, new, :, :n % ps] = a[:, old, :, :n % ps]
            refs[old] -= 1
            refs[new] = 1
            table[s][n // ps] = new
        lens[s] = n + c
        while _up(n, ps) < _up(lens[s], ps):
            new = free.pop(0)
            table[s][_up(n, ps)] = new
            refs[new] = 1
            n = (_up(n, ps) + 1) * ps
        first = lens[s] - c
        done = 0
        while done < c:                                     # the part of the new tokens that lies on one page
            p, at = table[s][(first + done) // ps], (first + done) % ps
            take = min(ps - at, c - done)
            k[:, p, :, at:at + take] = st["k_new"][:, b, done:done + take].transpose(1, 2)
            v[:, p, :, at:at + take] = st["v_new"][:, b, done:done + take].transpose(1, 2)
            done += take
    return _answer(st, table, lens, refs, k, v)


def _exact_pages(case, st):
    ps = case["page"]
    table, lens, refs = _lists(st)
    for s in st["gone"].tolist():
        for j in range(_up(lens[s], ps)):
            refs[table[s][j]] -= 1
            table[s][j] = -1
        lens[s] = 0
    for a, b in zip(st["src"].tolist(), st["dst"].tolist()):
        table[b], lens[b] = list(table[a]), lens[a]
        for j in range(_up(lens[a], ps)):
            refs[table[a][j]] += 1
    n = sum(r > 0 for r in refs)
    come = [p for p in range(n, len(refs)) if refs[p] > 0]
    to = [p for p in range(n) if refs[p] == 0]
    name = {a: b for a, b in zip(come, to)}
    k, v = st["k"].clone(), st["v"].clone()
    for a, b in name.items():
        k[:, b], v[:, b] = st["k"][:, a], st["v"][:, a]
        refs[b], refs[a] = refs[a], 0
    table = [[name.get(p, p) for p in row] for row in table]
    return _answer(st, table, lens, refs, k, v)
