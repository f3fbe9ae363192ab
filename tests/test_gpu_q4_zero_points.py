"""4-bit products of weights at or next to their zero points, and of infinite
inputs: nothing cancels, whatever the number of rows."""
import numpy as np
import pytest

from test_gpu_q4 import close, make, on_gpu, reference

pytestmark = pytest.mark.gpu

ROWS = [1, 2, 3, 8, 9, 16, 24, 32]


@pytest.fixture(scope="module")
def ex():
    from gemm_exl3_gemv_b200 import exl3
    return exl3


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m", ROWS)
def test_weights_next_to_their_zero_points(ex, m, group):
    """Every third channel's weights are all zero (q = z): its results are exactly zero.  The others have one
    weight in sixteen a step away from its zero point, so that the sum of q x is far larger than the result;
    the error allowed is of the products (q - z) x alone, as everywhere."""
    rng = np.random.default_rng(m + group)
    for fp32, zero in ((True, True), (False, True), (True, False)):
        c = make(m, 1280, 240, group, seed=m + group, zero=zero)
        z = np.full((1280, 240), 8, np.int64) if c["zero"] is None else np.repeat(c["zero"].astype(np.int64), group, 0)
        step = np.where(rng.random((1280, 240)) < 1 / 16, np.where(z < 15, 1, -1), 0)
        step[:, ::3] = 0
        c["q"] = (z + step).astype(np.uint8)
        # of every size, and nearly all of one sign: sums of q x are large, and inexact in fp32
        c["x"] = (2.0 ** rng.uniform(-14, 8, (m, 1280)) * np.where(rng.random((m, 1280)) < 0.1, -1, 1)).astype(np.float16)
        y = on_gpu(ex, c, fp32=fp32)
        assert (y[:, ::3] == 0).all()
        close(y, *reference(c), fp32)


@pytest.mark.parametrize("m", ROWS)
def test_infinite_inputs(ex, m):
    """An infinite input makes a result infinite, with the weight's sign, or NaN where the weight is zero; the
    other rows have nothing of it."""
    c = make(m, 256, 48, 64, seed=m)
    row, k, value = m // 2, 77, -np.inf if m % 2 else np.inf
    keep = c["x"].copy()
    c["x"][row, k] = value
    y = on_gpu(ex, c, fp32=True).cpu().numpy()
    w = c["q"][k].astype(np.float64) - c["zero"][k // 64]
    with np.errstate(invalid="ignore"):
        want = np.where(w == 0, np.nan, value * w)
    assert (w == 0).any() and np.array_equal(y[row], want.astype(np.float32), equal_nan=True)
    others = [i for i in range(m) if i != row]
    c["x"] = keep
    ref, tol = reference(c)
    assert np.all(np.abs(y[others] - ref[others]) <= tol[others])
