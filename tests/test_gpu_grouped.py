"""GPU parity of the grouped products (q4k_gemv_grouped, q4k_gemv_grouped_q8,
q4k_f16_gemm_grouped) against f64 products of the fields (numpy).

Q4_K: with T = sum (|d sc q| + |dmin m|) |x| and U the same with the row's
largest |x| everywhere, |y - y_ref| <= (280 + k/128) 2^-23 T + 2^-48 U: x is
carried to 2^-22 |x| or 2^-50 max|x|, a superblock's 256 products add up in f32
(257 roundings, each within 2^-23 of the sum of magnitudes), S_j in 5, and each
of the k/256 superblocks adds two terms.  That bound holds for any input; on
random data the roundings do not line up, so the 2-norm of all errors is held
to 2^-18 of the 2-norm of the results as well (280 roundings of 2^-24 that add
like a random walk are 2^-20): a lost low half of x would leave 2^-13.
The fp16 form: k 2^-23 sum |w16| |x16|.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from block_quantized_decode_q4_amd import q4k, synth  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    q4k.load_library()
    yield


class Weights:
    """groups x n rows of Q4_K with their two terms in f64."""

    def __init__(self, rng, groups, n, k):
        f = synth.draw_fields(rng, groups * n, k // 256)
        f.q[:, :, 32:64] = 0                          # a sub-block of zero codes
        f.sc[0] = 63
        f.m[0] = 63
        f.q[0] = 15
        self.bytes = synth.pack(f)
        d = f.d_bits.view(np.float16).astype(np.float64)[:, :, None]
        dmin = f.dmin_bits.view(np.float16).astype(np.float64)[:, :, None]
        up = np.repeat(d * f.sc, 32, axis=2) * f.q
        down = np.repeat(dmin * f.m, 32, axis=2)
        self.w = (up - down).reshape(groups, n, k)
        self.mag = (up + down).reshape(groups, n, k)


def _offsets(sizes):
    return np.concatenate(([0], np.cumsum(sizes))).astype(np.int32)


def _i32(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def _gpu(kind, w, x, y, off, n, k, groups, rows, **kw):
    """x: f32 array, (q, d), or f16 array by kind."""
    y_d = torch.from_numpy(y).cuda()
    w_d = torch.from_numpy(w).cuda()
    if kind == "f16":
        q4k.q4k_f16_gemm_grouped(w_d, torch.from_numpy(x).cuda(), y_d, _i32(off), n, k, groups,
                                 rows, **kw)
    else:
        nb = q4k.q4k_gemv_grouped_ws(k, rows)
        ws = torch.full((nb,), 0xFF, dtype=torch.uint8, device="cuda")     # NaN patterns
        if kind == "f32":
            q4k.q4k_gemv_grouped(w_d, torch.from_numpy(x).cuda(), y_d, _i32(off), n, k, groups,
                                 rows, ws=ws, **kw)
        else:
            q, d = (torch.from_numpy(a).cuda() for a in x)
            q4k.q4k_gemv_grouped_q8(w_d, q, d, y_d, _i32(off), n, k, groups, rows, ws=ws, **kw)
    torch.cuda.synchronize()
    return y_d.cpu().numpy()


def _x_value(kind, x):
    """The f64 values that x stands for (Q8: d q, rounded to f32 as documented)."""
    if kind != "q8":
        return x.astype(np.float64)
    q, d = x
    return (q.reshape(q.shape[0], -1, 32).astype(np.float32) * d[:, :, None]).reshape(
        q.shape).astype(np.float64)


def _make_x(rng, kind, count, k, spread=0):
    x = rng.standard_normal((count, k)) * np.exp2(rng.integers(-spread, spread + 1, (count, k)))
    if kind == "f16":
        return x.astype(np.float16)
    if kind == "f32":
        return x.astype(np.float32)
    q = rng.integers(-127, 128, size=(count, k)).astype(np.int8)
    d = (rng.random((count, k // 32)) * np.exp2(rng.integers(-spread - 6, spread + 1,
                                                             (count, k // 32)))).astype(np.float32)
    return q, d


def _check(kind, W, x, off, xr, yr, y0, got, n, k, norm=True):
    """Every y row against its product; rows no position names unchanged."""
    xv = _x_value(kind, x)
    named = np.zeros(y0.shape[0], bool)
    refs, errs = [], []
    groups = len(off) - 1
    for g in range(groups):
        for p in range(off[g], off[g + 1]):
            if xr[p] < 0 or yr[p] < 0 or xr[p] >= xv.shape[0] or yr[p] >= y0.shape[0]:
                continue
            v = xv[xr[p]]
            ref = W.w[g] @ v
            T = W.mag[g] @ np.abs(v)
            if kind == "f16":
                tol = k * 2.0 ** -23 * T
            else:
                U = W.mag[g].sum(1) * np.abs(v).max()
                tol = (280 + k / 128) * 2.0 ** -23 * T + 2.0 ** -48 * U
            err = np.abs(got[yr[p]] - ref)
            assert (err <= tol + 2.0 ** -149).all(), (g, p, float((err / (tol + 1e-300)).max()))
            named[yr[p]] = True
            refs.append(ref)
            errs.append(err)
    assert np.array_equal(got[~named].view(np.uint32), y0[~named].view(np.uint32))
    if norm and refs:
        assert np.linalg.norm(errs) <= 2.0 ** -18 * np.linalg.norm(refs)


class Mirror:
    def __init__(self, rng, groups, n, k):
        w = (rng.standard_normal((groups, n, k)) * 0.05).astype(np.float16)
        self.bytes = w
        self.w = w.astype(np.float64)
        self.mag = np.abs(self.w)


SIZES = [
    ([1], 1, 256), ([1], 16, 4096), ([0, 3, 0, 0, 1], 33, 512), ([16, 17, 0, 1], 50, 768),
    ([5] * 9, 130, 1280), ([40, 0, 100, 3], 257, 2048), ([1] * 70, 20, 256),
    ([0] * 63 + [2, 1, 33] + [0] * 70, 17, 512), ([200], 300, 1024), ([0, 0, 2], 1000, 2304),
]


# enough tiles for every way of cutting rows and k: few positions a group (four
# row tiles a wave), many (eight), the last with one, two and four waves along k
SIZES += [
    ([2] * 40, 450, 768), ([1, 0, 3] * 20, 600, 256), ([10] * 20, 1000, 256),
    ([9, 12] * 10, 1010, 512), ([17, 3, 8] * 7, 1500, 768), ([8] * 20, 840, 1280),
    ([30, 5] * 10, 700, 1024),
]
# the cut that the number of tiles decides: the coarse one, the fine one, and one
# where fewer tiles are there than the sizes allow
SIZES += [([40, 8], 20500, 256), ([40, 8], 4100, 512), ([0, 0, 70, 0, 0, 1], 5000, 1280)]
# few rows, up to two a group on average: with two and with four row tiles a wave
SIZES += [([1, 1], 9000, 512), ([3, 1, 0, 2], 5000, 768), ([1] * 8, 2100, 1280),
          ([9, 4, 0, 1, 0, 0, 0, 0], 40, 1024), ([2], 70, 256), ([16] + [0] * 7, 100, 2048),
          ([1, 1], 30, 8448)]


@pytest.mark.parametrize("kind", ["f32", "q8", "f16"])
@pytest.mark.parametrize("sizes,n,k", SIZES)
def test_grouped_sizes(kind, sizes, n, k):
    rng = np.random.default_rng(sum(sizes) + n + k)
    groups, rows = len(sizes), sum(sizes)
    W = (Mirror if kind == "f16" else Weights)(rng, groups, n, k)
    x = _make_x(rng, kind, rows, k)
    off = _offsets(sizes)
    y0 = np.full((rows, n), 123.25, np.float32)
    print("grouped %s sizes=%s n=%d k=%d" % (kind, sizes[:8], n, k), flush=True)
    got = _gpu(kind, W.bytes, x, y0, off, n, k, groups, rows)
    _check(kind, W, x, off, np.arange(rows), np.arange(rows), y0, got, n, k)


@pytest.mark.parametrize("sizes,n,k", [
    ([5, 0, 70], 130, 64), ([33, 64, 65, 1], 300, 320), ([400], 200, 256), ([1024], 520, 512),
    ([31, 0, 33], 65, 2048), ([64, 129, 2], 1100, 768)])
def test_grouped_f16_steps_of_k(sizes, n, k):
    """Long and short steps along k, tiles of 32 and 64 rows, ragged ends."""
    rng = np.random.default_rng(n + k)
    groups, rows = len(sizes), sum(sizes)
    W = Mirror(rng, groups, n, k)
    x = _make_x(rng, "f16", rows, k)
    off = _offsets(sizes)
    y0 = np.full((rows, n), 123.25, np.float32)
    print("grouped f16 steps sizes=%s n=%d k=%d" % (sizes, n, k), flush=True)
    got = _gpu("f16", W.bytes, x, y0, off, n, k, groups, rows)
    _check("f16", W, x, off, np.arange(rows), np.arange(rows), y0, got, n, k)


def test_grouped_f16_wide_tiles():
    """Shapes that take the 128-row tiles (groups of about a tile or more and
    enough of them), ragged in rows and columns; of 256 columns (the third) and of
    192 (the last)."""
    rng = np.random.default_rng(14)
    for sizes, n, k in (([300, 0, 5, 190], 8229, 128), ([129, 128, 127], 12300, 192),
                        ([200], 32700, 64), ([200], 16400, 64)):
        groups, rows = len(sizes), sum(sizes)
        w = torch.randn((groups, n, k), generator=torch.Generator("cuda").manual_seed(n),
                        device="cuda").mul_(0.05).half()
        x = rng.standard_normal((rows, k)).astype(np.float16)
        off = _offsets(sizes)
        print("grouped f16 wide sizes=%s n=%d k=%d" % (sizes, n, k), flush=True)
        y = torch.full((rows, n), float("nan"), device="cuda")
        perm = torch.from_numpy(rng.permutation(rows).astype(np.int32)).cuda()
        q4k.q4k_f16_gemm_grouped(w, torch.from_numpy(x).cuda(), y, _i32(off), n, k, groups, rows,
                                 y_rows=perm)
        got = y.cpu().numpy()[perm.cpu().numpy()]
        wf = w.cpu().numpy().astype(np.float64)
        for g in range(groups):
            part = slice(off[g], off[g + 1])
            ref = x[part].astype(np.float64) @ wf[g].T
            tol = k * 2.0 ** -23 * (np.abs(x[part].astype(np.float64)) @ np.abs(wf[g]).T)
            assert (np.abs(got[part] - ref) <= tol).all()


@pytest.mark.parametrize("kind", ["f32", "q8", "f16"])
def test_grouped_rows_gathered_scattered_and_left_out(kind):
    """Offsets that leave positions before and behind the groups, x by token,
    y scattered, rows out of range on either side."""
    rng = np.random.default_rng(8)
    n, k, groups, rows, x_count, y_count = 70, 512, 5, 60, 13, 75
    W = (Mirror if kind == "f16" else Weights)(rng, groups, n, k)
    x = _make_x(rng, kind, x_count, k)
    off = np.array([4, 20, 20, 41, 50, 53], np.int32)
    x_rows = rng.integers(0, x_count * 3, size=rows).astype(np.int32)
    x_rows[[7, 30]] = -1
    x_rows[[8, 42]] = x_count * 3                     # / 3: one beyond
    x_rows[31] = 2 ** 31 - 1
    y_rows = rng.permutation(y_count)[:rows].astype(np.int32)
    y_rows[[9, 33]] = -5
    y_rows[[10, 43]] = y_count
    y0 = np.full((y_count, n), -3.5, np.float32)
    got = _gpu(kind, W.bytes, x, y0, off, n, k, groups, rows, x_rows=_i32(x_rows), x_div=3,
               x_count=x_count, y_rows=_i32(y_rows), y_count=y_count)
    xr = np.where(x_rows < 0, -1, x_rows // 3)
    _check(kind, W, x, off, xr, y_rows, y0, got, n, k)


@pytest.mark.parametrize("kind", ["f32", "f16"])
def test_grouped_bad_offsets_stay_inside(kind):
    """Offsets that decrease, or lie outside the rows, give no access outside:
    the groups are cut to the rows.  Positions that two groups claim get either
    product or neither; a group apart from the others is as it should be."""
    rng = np.random.default_rng(9)
    n, k, groups, rows = 20, 256, 5, 14
    W = (Mirror if kind == "f16" else Weights)(rng, groups, n, k)
    x = _make_x(rng, kind, rows, k)
    y0 = np.full((rows + 2, n), 5.0, np.float32)
    off = np.array([-7, 3, 2, 6, 10, 1000], np.int32)
    got = _gpu(kind, W.bytes, x, y0, off, n, k, groups, rows, y_count=rows)
    assert (got[rows:] == 5.0).all()
    for g, lo, hi in ((3, 6, 10), (4, 10, 14)):
        for p in range(lo, hi):
            v = x[p].astype(np.float64)
            err = np.abs(got[p] - W.w[g] @ v)
            assert (err <= 300 * 2.0 ** -23 * (W.mag[g] @ np.abs(v)) + 1e-30).all(), (g, p)


def test_grouped_ranges_of_x():
    """Elements far apart in one row, rows near the ends of the f32 range, rows
    of zeros, and non-finite rows that leave the others alone."""
    rng = np.random.default_rng(10)
    n, k, groups, rows = 40, 1024, 2, 10
    W = Weights(rng, groups, n, k)
    x = _make_x(rng, "f32", rows, k, spread=20)
    x[1] *= np.float32(1e25)
    x[2] *= np.float32(1e-38)
    x[3] = 0.0
    x[4] = 1e-45
    x[5, 10] = 1e30
    x[6, 3] = np.inf
    x[7, 900] = np.nan
    off = _offsets([8, 2])
    y0 = np.full((rows, n), 1.0, np.float32)
    got = _gpu("f32", W.bytes, x, y0, off, n, k, groups, rows)
    assert not np.isfinite(got[6]).any() and not np.isfinite(got[7]).any()
    assert (got[3] == 0).all()
    keep = [0, 1, 2, 3, 4, 5, 8, 9]
    yr = np.where(np.isin(np.arange(rows), keep), np.arange(rows), -1)
    y1 = y0.copy()
    y1[[6, 7]] = got[[6, 7]]
    _check("f32", W, x, off, np.arange(rows), yr, y1, got, n, k, norm=False)


@pytest.mark.parametrize("kind", ["f32", "q8"])
@pytest.mark.parametrize("sizes,n", [([4, 1, 0, 2, 3], 40), ([2, 1, 0, 2, 3], 9000)])
def test_grouped_few_rows_ranges_of_x(kind, sizes, n):
    """Few rows, whose superblocks lie far apart, in either order: the largest
    first, last, and zeros between; non-finite ones leave other rows alone."""
    rng = np.random.default_rng(12)
    k, groups, rows = 2304, len(sizes), sum(sizes)
    W = Weights(rng, groups, n, k)
    x = _make_x(rng, kind, rows, k)
    scale = x if kind == "f32" else x[1]                 # what carries the range
    per = scale.shape[1] // 9
    up = np.array([-120, -60, -1000, -40, 0, 3, -1000, 40, 80], np.float64)
    for i, e in enumerate((up, up[::-1], rng.permutation(up), np.full(9, -1000.0))):
        scale[i] *= np.repeat(np.exp2(e), per).astype(np.float32)
    scale[4, per + 1] = np.inf
    scale[5, 8 * per + 3] = np.nan
    if kind == "q8":
        x[0][4, 256:512] = 5
        x[0][5, 2048:] = 5
    off = _offsets(sizes)
    y0 = np.full((rows, n), 1.0, np.float32)
    print("grouped few rows %s n=%d" % (kind, n), flush=True)
    got = _gpu(kind, W.bytes, x, y0, off, n, k, groups, rows)
    assert not np.isfinite(got[4]).any() and not np.isfinite(got[5]).any()
    assert (got[3] == 0).all()
    yr = np.where(np.isin(np.arange(rows), [4, 5]), -1, np.arange(rows))
    y1 = y0.copy()
    y1[[4, 5]] = got[[4, 5]]
    _check(kind, W, x, off, np.arange(rows), yr, y1, got, n, k, norm=False)


def test_grouped_weights_not_finite_stay_in_their_row():
    rng = np.random.default_rng(11)
    W = Weights(rng, 1, 40, 512)
    w = W.bytes.copy().reshape(40, 2, 144)
    w[5, 1, 0:2] = np.array([0x00, 0x7E], np.uint8)   # d = NaN
    w[9, 0, 2:4] = np.array([0x00, 0x7C], np.uint8)   # dmin = inf
    x = _make_x(rng, "f32", 3, 512)
    y0 = np.zeros((3, 40), np.float32)
    got = _gpu("f32", w.reshape(-1), x, y0, _offsets([3]), 40, 512, 1, 3)
    ok = np.ones(40, bool)
    ok[[5, 9]] = False
    assert not np.isfinite(got[:, [5, 9]]).any()
    ref = x.astype(np.float64) @ W.w[0].T
    T = np.abs(x.astype(np.float64)) @ W.mag[0].T
    assert (np.abs(got - ref)[:, ok] <= 300 * 2.0 ** -23 * T[:, ok]).all()


def test_grouped_same_bits_each_time():
    rng = np.random.default_rng(12)
    W = Weights(rng, 3, 200, 1536)
    x = _make_x(rng, "f32", 30, 1536)
    y0 = np.zeros((30, 200), np.float32)
    off = _offsets([20, 0, 10])
    a = _gpu("f32", W.bytes, x, y0, off, 200, 1536, 3, 30)
    b = _gpu("f32", W.bytes, x, y0, off, 200, 1536, 3, 30)
    assert np.array_equal(a.view(np.uint32), b.view(np.uint32))
    # a position's result does not depend on who shares its tile
    c = _gpu("f32", W.bytes, x[:5], y0[:5], _offsets([5, 0, 0]), 200, 1536, 3, 5)
    np.testing.assert_allclose(c, a[:5], rtol=0, atol=2e-4 * np.abs(a).max())


@pytest.mark.parametrize("kind", ["f32", "f16"])
def test_grouped_offsets_that_name_more_tiles_than_32_bits(kind):
    """Every second group claims all the rows: 4096 groups of 2^21 rows, which
    the grid does not hold; the rows around y stay."""
    n, groups, rows = 1024, 8192, 2 ** 21
    k = 256 if kind == "f32" else 64
    off = torch.zeros(groups + 1, dtype=torch.int32, device="cuda")
    off[1::2] = rows
    y = torch.full((3, n), 5.0, device="cuda")
    if kind == "f32":
        w = torch.zeros((groups * n, 144), dtype=torch.uint8, device="cuda")
        ws = torch.empty(q4k.q4k_gemv_grouped_ws(k, rows), dtype=torch.uint8, device="cuda")
        q4k.q4k_gemv_grouped(w, torch.ones((1, k), device="cuda"), y, off, n, k, groups, rows,
                             x_count=1, y_count=1, ws=ws)
    else:
        w = torch.zeros((groups * n, k), dtype=torch.float16, device="cuda")
        q4k.q4k_f16_gemm_grouped(w, torch.ones((1, k), dtype=torch.float16, device="cuda"), y,
                                 off, n, k, groups, rows, x_count=1, y_count=1)
    torch.cuda.synchronize()
    assert (y[1:] == 5.0).all()
