"""The grouped Q4_K products' one-launch form (few rows, up to two a group, with
two and with four row tiles a wave): positions left out, rows out of range,
offsets that decrease, weights that are not finite.  References and bounds are
those of test_gpu_grouped.py."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from block_quantized_decode_q4_amd import q4k  # noqa: E402
from test_gpu_grouped import Weights, _check, _gpu, _i32, _make_x, _x_value  # noqa: E402

pytestmark = pytest.mark.gpu

GROUPS, ROWS = 5, 8
SHAPES = [(40, 512), (9000, 512), (33, 2304)]       # two, four and two row tiles a wave


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    q4k.load_library()
    yield


@pytest.mark.parametrize("kind", ["f32", "q8"])
@pytest.mark.parametrize("n,k", SHAPES)
@pytest.mark.parametrize("off", [[1, 3, 3, 6, 7, 8], [0, 8, 8, 8, 8, 8], [0, 0, 0, 0, 0, 7],
                                 [0, 0, 0, 0, 0, 0]])
def test_positions_left_out(kind, n, k, off):
    """x by token, y scattered, rows out of range on either side; x row 0, which
    no position takes, is not finite."""
    rng = np.random.default_rng(n + k + off[1])
    W = Weights(rng, GROUPS, n, k)
    x_count, y_count = 5, 11
    x = _make_x(rng, kind, x_count, k)
    (x if kind == "f32" else x[1])[0, :2] = [np.nan, np.inf]
    for bad in range(4):
        x_rows = rng.integers(3, x_count * 3, size=ROWS).astype(np.int32)
        y_rows = rng.permutation(y_count)[:ROWS].astype(np.int32)
        at = rng.permutation(ROWS)
        x_rows[at[: bad + 1]] = [-1, x_count * 3, 2 ** 31 - 1, -2 ** 31][: bad + 1]
        y_rows[at[4: 4 + bad]] = [-5, y_count, 2 ** 31 - 1][:bad]
        y0 = np.full((y_count, n), -3.5, np.float32)
        print("grouped few, left out %s n=%d k=%d off=%s x=%s y=%s" % (kind, n, k, off, x_rows, y_rows),
              flush=True)
        got = _gpu(kind, W.bytes, x, y0, np.array(off, np.int32), n, k, GROUPS, ROWS,
                   x_rows=_i32(x_rows), x_div=3, x_count=x_count, y_rows=_i32(y_rows),
                   y_count=y_count)
        xr = np.where(x_rows < 0, -1, x_rows // 3)
        _check(kind, W, x, off, xr, y_rows, y0, got, n, k)


@pytest.mark.parametrize("kind", ["f32", "q8"])
@pytest.mark.parametrize("n,k", SHAPES)
def test_offsets_that_decrease_stay_inside(kind, n, k):
    """Positions that two groups claim get either product; groups apart from the
    others are as they should be, and so are the rows behind the last."""
    rng = np.random.default_rng(n + k)
    W = Weights(rng, GROUPS, n, k)
    x = _make_x(rng, kind, ROWS, k)
    y0 = np.full((ROWS + 2, n), 5.0, np.float32)
    off = np.array([-7, 3, 2, 6, 7, 1000], np.int32)
    print("grouped few, offsets %s n=%d k=%d" % (kind, n, k), flush=True)
    got = _gpu(kind, W.bytes, x, y0, off, n, k, GROUPS, ROWS, y_count=ROWS)
    assert (got[ROWS:] == 5.0).all()
    xv = _x_value(kind, x)
    for g, p in ((3, 6), (4, 7)):
        T = W.mag[g] @ np.abs(xv[p])
        U = W.mag[g].sum(1) * np.abs(xv[p]).max()
        tol = (280 + k / 128) * 2.0 ** -23 * T + 2.0 ** -48 * U
        assert (np.abs(got[p] - W.w[g] @ xv[p]) <= tol).all(), (g, p)


@pytest.mark.parametrize("kind", ["f32", "q8"])
@pytest.mark.parametrize("n,k", SHAPES)
def test_weights_not_finite_stay_in_their_row(kind, n, k):
    rng = np.random.default_rng(n + k + 1)
    W = Weights(rng, GROUPS, n, k)
    w = W.bytes.copy().reshape(GROUPS, n, k // 256, 144)
    w[1, 5, 1, 0:2] = np.array([0x00, 0x7E], np.uint8)     # d = NaN
    w[1, 9, 0, 2:4] = np.array([0x00, 0x7C], np.uint8)     # dmin = inf
    w[3, 20, 0, 0:2] = np.array([0x00, 0x7C], np.uint8)    # d = inf
    x = _make_x(rng, kind, ROWS, k)
    off = np.array([0, 2, 5, 5, 7, 8], np.int32)
    y0 = np.zeros((ROWS, n), np.float32)
    print("grouped few, weights %s n=%d k=%d" % (kind, n, k), flush=True)
    got = _gpu(kind, w.reshape(-1), x, y0, off, n, k, GROUPS, ROWS)
    assert not np.isfinite(got[2:5][:, [5, 9]]).any() and not np.isfinite(got[5:7, 20]).any()
    bad = ~np.isfinite(got)
    assert bad.sum() == 3 * 2 + 2
    for g, p in ((0, 0), (0, 1), (1, 2), (1, 3), (1, 4), (3, 5), (3, 6), (4, 7)):
        v = _x_value(kind, x)[p]
        U = W.mag[g].sum(1) * np.abs(v).max()
        tol = (280 + k / 128) * 2.0 ** -23 * (W.mag[g] @ np.abs(v)) + 2.0 ** -48 * U
        assert (np.abs(got[p] - W.w[g] @ v) <= tol)[~bad[p]].all(), (g, p)
