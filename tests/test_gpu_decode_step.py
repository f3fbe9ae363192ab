"""The cache, the attention and the 4-bit products together, as a server uses
them: prompts are taken in, a sequence is forked, drafted tokens are verified and
partly dropped, a sequence leaves and the pool is compacted, step after step.
Every step's attention and every projection is checked in fp64 against a model
that keeps plain lists of tokens."""
import numpy as np
import pytest

import cache_model

pytestmark = pytest.mark.gpu

HID, HEADS, KV, D, GROUP = 256, 4, 2, 64, 64


class Layer:
    """q, k, v and o with 4-bit weights: on the GPU, and in fp64."""

    def __init__(self, ex, seed):
        import torch
        rng = np.random.default_rng(seed)
        self.ex, self.gpu, self.w = ex, {}, {}
        for name, k, n in (("q", HID, HEADS * D), ("k", HID, KV * D), ("v", HID, KV * D), ("o", HEADS * D, HID)):
            q = rng.integers(0, 16, (k, n)).astype(np.uint8)
            scale = (rng.uniform(0.5, 1.5, (k // GROUP, n)) / np.sqrt(k) / 4).astype(np.float16)
            zero = rng.integers(6, 10, (k // GROUP, n)).astype(np.uint8)
            dev = lambda a: torch.from_numpy(a).cuda()
            self.gpu[name] = (ex.q4_pack(dev(q)), dev(scale), dev(zero))
            self.w[name] = (q.astype(np.float64) - np.repeat(zero.astype(np.float64), GROUP, 0)) * \
                np.repeat(scale.astype(np.float64), GROUP, 0)

    def gemm(self, name, x, ws):
        return self.ex.q4_gemm(x, *self.gpu[name], GROUP, workspace=ws)

    def close(self, name, x, y):
        x, y = x.double().cpu().numpy(), y.double().cpu().numpy()
        ref = x @ self.w[name]
        tol = (x.shape[1] / 16 + 24) * 2.0 ** -22 * (np.abs(x) @ np.abs(self.w[name])) + 2.0 ** -11 * np.abs(ref) + 2.0 ** -25
        assert np.all(np.abs(y - ref) <= tol), name


def test_serving_steps():
    import torch
    from gemm_exl3_gemv_b200 import exl3 as ex
    from gemm_exl3_gemv_b200.kvcache import KvCache
    layers = [Layer(ex, 20 + i) for i in range(2)]
    cache = KvCache.empty(2, 60, KV, 16, D, 6, 10)
    ids = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    tokens = {s: [([], []) for _ in layers] for s in range(6)}          # per layer: keys, values
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    ws = cache.attention_workspace(4, 32, HEADS)
    ws = torch.zeros(max(ws.numel(), ex.q4_workspace_bytes(32, HID, HID)), dtype=torch.uint8, device="cuda")

    def step(seqs, counts, window=0, sinks=0):
        """Every layer of a step for these sequences, counts new tokens each (padded to the longest)."""
        m, n = max(counts), len(seqs)
        s, c = ids(seqs), ids(counts)
        cache.extend(s, m, counts=c)
        for li, layer in enumerate(layers):
            x = torch.randn(n * m, HID, generator=gen, device="cuda").half()
            q, k, v = (torch.cat([layer.gemm(w, part, ws) for part in x.split(32)]) for w in "qkv")
            for w, y in zip("qkv", (q, k, v)):
                layer.close(w, x, y)
            cache.write(li, s, k.view(n, m, KV, D), v.view(n, m, KV, D), counts=c)
            for b, seq in enumerate(seqs):
                for kept, y in zip(tokens[seq][li], (k, v)):
                    kept += list(y.view(n, m, KV, D)[b, :counts[b]].double().cpu().numpy())
            if m > 32:
                continue                                                # a prompt: its attention is not this call's
            att = cache.attention(li, s, q.view(n, m, HEADS, D), counts=c, window=window, sinks=sinks, workspace=ws)
            for b, seq in enumerate(seqs):
                keys, values = (np.array(t) for t in tokens[seq][li])
                ref, _, tol, _ = cache_model.attention(q.view(n, m, HEADS, D)[b, :counts[b]].double().cpu().numpy(), keys,
                                                       values, len(keys) - counts[b], D ** -0.5, window, sinks)
                got = att[b, :counts[b]].double().cpu().numpy()
                assert np.all(np.abs(got - ref) <= tol), (li, seq)
            rows = att.view(n * m, HEADS * D)
            y = torch.cat([layer.gemm("o", part, ws) for part in rows.split(32)])
            layer.close("o", rows, y)

    def keep(seqs, lens):
        cache.truncate(ids(seqs), ids(lens))
        for s, n in zip(seqs, lens):
            for kept in tokens[s]:
                for t in kept:
                    del t[n:]

    step([0, 2, 4], [40, 75, 9])                        # prompts
    step([4, 0, 2], [1, 1, 1])                          # decode
    cache.fork(ids([2]), ids([5]))
    tokens[5] = [tuple(list(t) for t in kept) for kept in tokens[2]]
    step([5, 0, 2, 4], [8, 8, 5, 1])                    # drafted tokens; the forked sequences part
    keep([5, 2, 0], [79, 77, 41])                       # some are accepted
    step([0, 5], [1, 1], window=20, sinks=2)
    keep([0], [0])                                      # one leaves
    cache.compact()
    step([2, 4, 5], [32, 3, 17], window=50, sinks=4)
    step([3], [25])                                     # a new one
    step([3, 5, 4, 2], [1, 1, 1, 1])
    cache.check()
    assert cache.lens.tolist() == [len(tokens[s][0][0]) for s in range(6)]
    assert ex.workspace_status(ws) == ex.EXL3_OK


def test_a_stream_given_gets_its_own_memory():
    """Calls on a stream that is given, with the results, workspaces and the cache made by the calls, while the
    current stream is busy and memory that is handed out again holds ones."""
    import torch
    from gemm_exl3_gemv_b200 import exl3 as ex
    from gemm_exl3_gemv_b200.kvcache import KvCache
    rng = np.random.default_rng(31)
    dev = lambda a: torch.from_numpy(a).cuda()
    x, q = rng.standard_normal((12, 2048)).astype(np.float16), rng.integers(0, 16, (2048, 128)).astype(np.uint8)
    scale = rng.uniform(0.01, 0.02, (32, 128)).astype(np.float16)
    k, v, qq = (rng.standard_normal((1, 600 if i < 2 else 4, 2, 128)).astype(np.float16) for i in range(3))
    gx, gq, gs, gk, gv, gqq, ids = dev(x), dev(q), dev(scale), dev(k), dev(v), dev(qq), torch.zeros(1, dtype=torch.int32, device="cuda")
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        ones = [torch.full((n,), -1, dtype=torch.int32, device="cuda") for n in (1 << 16, 1 << 20, 1 << 22)]
    torch.cuda.synchronize()
    del ones
    torch.cuda._sleep(100_000_000)                        # some 50 ms of the current stream
    c = KvCache.empty(1, 16, 2, 64, 128, 1, 12, stream=stream)
    c.extend(ids, 600, stream=stream)
    c.write(0, ids, gk, gv, stream=stream)
    att = c.attention(0, ids, gqq, stream=stream)
    ys = [ex.q4_gemm(gx[:m], ex.q4_pack(gq, stream=stream), gs, None, 64, fp32=True, stream=stream) for m in (1, 12)]
    stream.synchronize()
    got, gys = att.double().cpu().numpy()[0], [y.double().cpu().numpy() for y in ys]
    assert c.status(stream) == ex.EXL3_OK
    w = (q.astype(np.float64) - 8) * np.repeat(scale.astype(np.float64), 64, 0)
    for m, y in zip((1, 12), gys):                        # 2048 inputs in fp32: 152 steps of 2^-22 of the magnitudes
        assert np.all(np.abs(y - x[:m].astype(np.float64) @ w) <= 152 * 2.0 ** -22 * (np.abs(x[:m].astype(np.float64)) @ np.abs(w)))
    ref, _, tol, _ = cache_model.attention(qq[0].astype(np.float64), k[0].astype(np.float64), v[0].astype(np.float64), 596, 128 ** -0.5)
    assert np.all(np.abs(got - ref) <= tol)
