"""exl3_q4_gemm and exl3_q4_pack on the GPU against an fp64 evaluation of the
definition from the unpacked values."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    from gemm_exl3_gemv_b200 import exl3
    return exl3


def make(m, k, n, group, seed, zero=True):
    rng = np.random.default_rng(seed)
    return dict(x=rng.standard_normal((m, k)).astype(np.float16), q=rng.integers(0, 16, (k, n)).astype(np.uint8),
                scale=(rng.uniform(0.5, 1.5, (k // group, n)) / np.sqrt(k) / 4).astype(np.float16),
                zero=rng.integers(0, 16, (k // group, n)).astype(np.uint8) if zero else None, group=group)


def reference(c):
    """The product in fp64, and the error allowed: the operands' products are
    exact in fp32 (11 bits times 5), a sum over k inputs takes at most k/16 + 24
    steps (16 inputs a step, the groups, warps and CTAs behind them), each off
    by at most 2^-22 of the sum of magnitudes; scaling rounds once more."""
    x, g = c["x"].astype(np.float64), c["group"]
    z = 8 if c["zero"] is None else np.repeat(c["zero"].astype(np.float64), g, 0)
    w = (c["q"].astype(np.float64) - z) * np.repeat(c["scale"].astype(np.float64), g, 0)
    return x @ w, (x.shape[1] / 16 + 24) * 2.0 ** -22 * (np.abs(x) @ np.abs(w))


def on_gpu(ex, c, **kw):
    import torch
    d = {k: torch.from_numpy(v).cuda() for k, v in c.items() if isinstance(v, np.ndarray)}
    return ex.q4_gemm(d["x"], ex.q4_pack(d["q"]), d["scale"], d.get("zero"), c["group"], **kw)


def close(y, ref, tol, fp32):
    y = y.double().cpu().numpy()
    if not fp32:
        tol = tol + 2.0 ** -11 * np.abs(ref) + 2.0 ** -25          # half a step of fp16
    assert np.all(np.abs(y - ref) <= tol), np.max(np.abs(y - ref) / tol)


SHAPES = [(64, 16, 32), (64, 16, 64), (128, 48, 128), (192, 80, 64), (256, 384, 32), (1088, 144, 64), (5120, 1024, 128)]


@pytest.mark.parametrize("k,n,group", SHAPES)
@pytest.mark.parametrize("m", [1, 2, 7, 8, 9, 16, 17, 31, 32])
def test_q4_matches_definition(ex, m, k, n, group):
    for fp32 in (True, False):
        c = make(m, k, n, group, seed=m + k + n, zero=(m + n) % 3 != 0)
        y = on_gpu(ex, c, fp32=fp32)
        assert y.shape == (m, n)
        close(y, *reference(c), fp32)


@pytest.mark.parametrize("m,k,n", [(1, 17408, 5120), (32, 5120, 17408), (5, 128, 33008)])
def test_q4_large(ex, m, k, n):
    c = make(m, k, n, 128, seed=9)
    close(on_gpu(ex, c, fp32=True), *reference(c), True)


@pytest.mark.parametrize("group", [32, 64])
@pytest.mark.parametrize("m", [2, 8, 16, 24, 32])
def test_q4_narrow_and_deep(ex, m, group):
    """Few channels and many inputs, cut as finely as it goes along the inputs: at the most rows of a kernel
    shape the stages of the rings are at their largest."""
    for k, n in ((8192, 64), (4160, 272)):
        c = make(m, k, n, group, seed=m + n)
        close(on_gpu(ex, c, fp32=True), *reference(c), True)


@pytest.mark.parametrize("m,k,n,group", [(9, 192, 33008, 64), (32, 128, 38016, 32), (12, 65536, 16, 128), (32, 64, 2048, 64),
                                         (25, 4160, 4112, 32), (16, 128, 128, 128)])
def test_q4_many_rows_extremes(ex, m, k, n, group):
    """More blocks of channels than the GPU has places, one block of many inputs, one stage of inputs (or half
    of one), a last block and a last stage that are not full."""
    c = make(m, k, n, group, seed=m + 3 * group, zero=m != 32)
    close(on_gpu(ex, c, fp32=True), *reference(c), True)


def test_q4_one_workspace_for_any_rows(ex):
    """The workspace for 32 rows serves every number of rows, one product after the other."""
    import torch
    c = make(32, 1024, 4096, 64, seed=23)
    d = {k: torch.from_numpy(v).cuda() for k, v in c.items() if isinstance(v, np.ndarray)}
    packed, ws = ex.q4_pack(d["q"]), ex.q4_alloc_workspace(32, 1024, 4096)
    ref, tol = reference(c)
    for m in (32, 1, 24, 8, 9, 2, 17, 16, 32):
        close(ex.q4_gemm(d["x"][:m], packed, d["scale"], d["zero"], 64, fp32=True, workspace=ws), ref[:m], tol[:m], True)


def test_q4_side_by_side_on_streams(ex):
    """Products of all three kernels on streams of their own: each as alone."""
    import torch
    cases = [make(32, 2048, 4096, 128, seed=24), make(12, 4096, 1024, 64, seed=25), make(3, 2048, 2048, 32, seed=26)]
    dev = [{k: torch.from_numpy(v).cuda() for k, v in c.items() if isinstance(v, np.ndarray)} for c in cases]
    packed = [ex.q4_pack(d["q"]) for d in dev]
    ws = [ex.q4_alloc_workspace(c["x"].shape[0], *c["q"].shape) for c in cases]
    call = lambda i: ex.q4_gemm(dev[i]["x"], packed[i], dev[i]["scale"], dev[i]["zero"], cases[i]["group"], fp32=True, workspace=ws[i])
    alone = [call(i) for i in range(3)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(3)], [[], [], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(call(i))
    torch.cuda.synchronize()
    for i, c in enumerate(cases):
        close(alone[i], *reference(c), True)
        assert all(torch.equal(y, alone[i]) for y in got[i])


def test_q4_pack_layout(ex):
    """Every word of the packed tiles, field by field from the documented layout."""
    import torch
    q = np.random.default_rng(3).integers(0, 256, (192, 32)).astype(np.uint8)     # high bits are not taken
    got = ex.q4_pack(torch.from_numpy(q).cuda()).cpu().numpy().view(np.uint32)
    assert got.shape == (2, 3, 32, 4)
    for tn, tk, g, t, j in np.ndindex(2, 3, 8, 4, 4):
        word = sum(int(q[64 * tk + 32 * (j // 2) + 8 * t + 4 * (j % 2) + i, 16 * tn + g + 8 * c] & 15) <<
                   (4 * c + 8 * (i // 2) + 16 * (i % 2)) for c in range(2) for i in range(4))
        assert got[tn, tk, 4 * g + t, j] == word


def test_q4_one_row_and_given_buffers(ex):
    import torch
    c = make(1, 256, 64, 64, seed=4)
    ref, tol = reference(c)
    d = {k: torch.from_numpy(v).cuda() for k, v in c.items() if isinstance(v, np.ndarray)}
    packed, ws = ex.q4_pack(d["q"]), ex.q4_alloc_workspace(1, 256, 64)
    out = torch.full((64,), float("nan"), dtype=torch.float32, device="cuda")
    y = ex.q4_gemm(d["x"][0], packed, d["scale"], d["zero"], 64, out=out, fp32=True, workspace=ws)
    assert y.shape == (64,) and y.data_ptr() == out.data_ptr()
    close(out, ref[0], tol[0], True)


def test_q4_rows_do_not_touch_each_other(ex):
    """A row of infinities and NaN stays in its own row; zeros beyond 15 are taken as they are."""
    import torch
    c = make(6, 128, 32, 64, seed=5)
    c["zero"][:] = 255
    c["x"][2] = np.inf
    c["x"][4] = np.nan
    y = on_gpu(ex, c, fp32=True).cpu()
    keep = [0, 1, 3, 5]
    c["x"] = c["x"][keep]
    ref, tol = reference(c)
    assert not torch.isfinite(y[[2, 4]]).any()
    close(y[keep], ref, tol, True)


@pytest.mark.parametrize("m", [1, 12, 32])
def test_q4_repeatable_and_shares_a_workspace(ex, m):
    """Bitwise repeatable, through a graph too; one workspace serves products of several shapes and the
    trellis products in any order."""
    import torch
    from gemm_exl3_gemv_b200 import synth
    from gpu_helpers import to_dev
    cases = [make(m, k, n, 64, seed=6 + k) for k, n in ((1024, 96), (128, 2048), (4096, 16))]
    dev = [{k: torch.from_numpy(v).cuda() for k, v in c.items() if isinstance(v, np.ndarray)} for c in cases]
    packed = [ex.q4_pack(d["q"]) for d in dev]
    spec = synth.MatrixSpec("q4ws", 256, 384, 3, m, seed=7)
    inp = synth.make_inputs(spec)
    tr = [to_dev(a) for a in (inp.x, inp.packed, inp.scale, inp.su, inp.sv)]
    need = max([ex.q4_workspace_bytes(m, *c["q"].shape) for c in cases] + [ex.workspace_bytes(m, 256, 384, 3)])
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")

    def step():
        ys = [ex.q4_gemm(d["x"], p, d["scale"], d["zero"], 64, fp32=True, workspace=ws) for d, p in zip(dev, packed)]
        return ys + [ex.gemm(*tr, 3, fp32=True, workspace=ws)]

    first = [y.clone() for y in step()]
    for c, y in zip(cases, first):
        close(y, *reference(c), True)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(step(), first))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ys = step()
    for _ in range(2):
        for y in ys:
            y.fill_(float("nan"))
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(ys, first))


@pytest.mark.parametrize("m", [2, 13, 31])
def test_q4_chained_products(ex, m):
    """A product's rows are another's inputs, right behind the packing of its weights; in a graph too."""
    import torch
    a, b = make(m, 1024, 640, 128, seed=20), make(m, 640, 208, 64, seed=21)
    dev = [{k: torch.from_numpy(v).cuda() for k, v in c.items() if isinstance(v, np.ndarray)} for c in (a, b)]
    ws = [ex.q4_alloc_workspace(m, 1024, 640), ex.q4_alloc_workspace(m, 640, 208)]

    def run():
        y = ex.q4_gemm(dev[0]["x"], ex.q4_pack(dev[0]["q"]), dev[0]["scale"], dev[0]["zero"], 128, workspace=ws[0])
        return y, ex.q4_gemm(y, ex.q4_pack(dev[1]["q"]), dev[1]["scale"], dev[1]["zero"], 64, fp32=True, workspace=ws[1])

    def check(y, z):
        close(y, *reference(a), False)
        close(z, *reference({**b, "x": y.cpu().numpy()}), True)

    check(*run())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run()
    for _ in range(2):
        dev[0]["x"].mul_(0.5)
        a["x"] = dev[0]["x"].cpu().numpy()
        g.replay()
        check(*out)


@pytest.mark.parametrize("m,k,group", [(12, 640, 64), (32, 5120, 128)])
def test_q4_withheld_inputs_time_out_and_report(ex, m, k, group):
    """x withheld through the workspace's injection word: the waits run out, the call ends and the status
    says so; the next call is right."""
    import torch
    c = make(m, k, 256, group, seed=22)
    d = {k: torch.from_numpy(v).cuda() for k, v in c.items() if isinstance(v, np.ndarray)}
    packed, ws = ex.q4_pack(d["q"]), ex.q4_alloc_workspace(m, k, 256)
    ws[4:8] = 1
    ex.q4_gemm(d["x"], packed, d["scale"], d["zero"], group, workspace=ws)
    assert ex.workspace_status(ws) == ex.EXL3_ERR_TIMEOUT
    ws[4:8] = 0
    close(ex.q4_gemm(d["x"], packed, d["scale"], d["zero"], group, fp32=True, workspace=ws), *reference(c), True)
    assert ex.workspace_status(ws) == ex.EXL3_OK


def test_q4_refusals(ex):
    import torch
    c = make(2, 128, 32, 64, seed=8)
    d = {k: torch.from_numpy(v).cuda() for k, v in c.items() if isinstance(v, np.ndarray)}
    packed = ex.q4_pack(d["q"])
    ok = dict(x=d["x"], packed=packed, scale=d["scale"], zero=d["zero"], group=64)
    bad_values = [dict(x=d["x"].float()), dict(x=d["x"].cpu()), dict(x=d["x"].t().contiguous().t()),
                  dict(scale=d["scale"][:1]), dict(zero=d["zero"].int()), dict(packed=packed.view(-1)),
                  dict(out=torch.empty(2, 16, device="cuda", dtype=torch.float16))]
    for change in bad_values:
        with pytest.raises(ValueError):
            ex.q4_gemm(**{**ok, **change})
    for change in (dict(group=96), dict(group=16), dict(x=d["x"].repeat(17, 1))):
        with pytest.raises(ex.Exl3Error) as e:
            ex.q4_gemm(**{**ok, **change})
        assert e.value.status == ex.EXL3_ERR_UNSUPPORTED
    with pytest.raises(ex.Exl3Error) as e:
        ex.q4_gemm(**ok, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == ex.EXL3_ERR_WORKSPACE
    with pytest.raises(ValueError):
        ex.q4_pack(d["q"].t())
    with pytest.raises(ex.Exl3Error):
        ex.q4_pack(torch.zeros(64, 24, dtype=torch.uint8, device="cuda"))
