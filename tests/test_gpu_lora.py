"""GPU parity of the low-rank adapters (q4k_lora) against f64 (numpy).

Every sum is f32: v = A x errs by (k + 1) 2^-23 of sum |A| |x|, times the
scale; v goes on as two binary16 numbers, which lose 2^-22 of it or 2^-39 of
its row's largest; B v and the base add r + 1 roundings more:
|y - y_ref| <= (k + r + 4) 2^-23 (|base| + |scale| sum_r |B| sum_k |A| |x|)
+ 2^-38 |scale| sum_r |B| max_r |A x|.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from block_quantized_decode_q4_amd import q4k  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    q4k.load_library()
    yield


def _group(ids, adapters):
    off = torch.empty(adapters + 1, dtype=torch.int32, device="cuda")
    order = torch.empty(len(ids), dtype=torch.int32, device="cuda")
    n = q4k.q4k_moe_group_ws(len(ids), adapters, 1)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    q4k.q4k_moe_group(torch.from_numpy(ids).cuda(), off, order, len(ids), adapters, ws=ws)
    return off, order


@pytest.mark.parametrize("rows,adapters,r,n,k,kind,ragged,base", [
    (1, 1, 1, 1, 8, "f32", False, "apart"), (1, 3, 16, 300, 512, "f16", False, "in place"),
    (5, 2, 8, 64, 40, "bf16", True, "apart"), (33, 4, 17, 131, 264, "f32", True, "none"),
    (70, 70, 64, 129, 1024, "f16", True, "apart"), (100, 3, 65, 67, 136, "f32", True, "in place"),
    (257, 5, 130, 260, 320, "bf16", False, "none"), (600, 2, 4, 1024, 256, "f16", True, "apart"),
    (40, 90, 6, 50, 72, "f32", True, "apart"), (3, 2, 1024, 20, 64, "f16", True, "apart"),
    # odd ranks and widths: pieces of B at its very end, rows of y on any element
    (2, 1, 1, 3, 8, "f16", False, "in place"), (9, 1, 3, 2, 64, "f32", False, "in place"),
    (37, 3, 7, 5, 128, "f16", False, "in place"), (600, 3, 61, 257, 256, "f16", True, "in place"),
    (4100, 2, 13, 259, 64, "f32", False, "in place"), (50, 2, 67, 1023, 128, "bf16", True, "apart"),
])
def test_lora(rows, adapters, r, n, k, kind, ragged, base):
    rng = np.random.default_rng(rows + adapters + r + n + k)
    ids = rng.integers(-1, adapters, size=rows).astype(np.int32)
    ids[0] = adapters - 1
    x = torch.from_numpy(rng.standard_normal((rows, k)).astype(np.float32)).to(TYPES[kind])
    a = (rng.standard_normal((adapters, r, k)) / np.sqrt(k)).astype(np.float16)
    b = (rng.standard_normal((adapters, n, r)) * 0.3).astype(np.float16)
    ranks = rng.integers(0, r + 1, size=adapters).astype(np.int32) if ragged else None
    if ragged:
        ranks[0] = 0
        ranks[-1] = r
        for i in range(adapters):                     # never read
            a[i, ranks[i]:] = np.nan
            b[i, :, ranks[i]:] = np.inf
        ranks[-1] = r + 5                             # cut to r
    scales = (0.5 + rng.random(adapters)).astype(np.float32) if ragged else None
    y0 = rng.standard_normal((rows, n)).astype(np.float32)
    base0 = rng.standard_normal((rows, n)).astype(np.float32)
    y = torch.from_numpy(y0).cuda()
    base_d = dict(apart=torch.from_numpy(base0).cuda(), none=None)
    base_d["in place"] = y
    off, order = _group(ids, adapters)
    ws = torch.full((q4k.q4k_lora_ws(rows, r),), 0xFF, dtype=torch.uint8, device="cuda")
    dev = [None if t is None else torch.from_numpy(t).cuda() for t in (ranks, scales)]
    print("lora rows=%d adapters=%d r=%d n=%d k=%d %s" % (rows, adapters, r, n, k, kind), flush=True)
    q4k.q4k_lora(x.cuda(), torch.from_numpy(a).cuda(), torch.from_numpy(b).cuda(), y, off, order, n,
                 k, r, adapters, rows, base=base_d[base], ranks=dev[0], scales=dev[1], ws=ws)
    got = y.cpu().numpy()
    start = {"apart": base0, "in place": y0, "none": np.zeros_like(y0)}[base].astype(np.float64)
    xv = x.float().numpy().astype(np.float64)
    for t in range(rows):
        i = ids[t]
        if i < 0:
            assert np.array_equal(got[t], y0[t])
            continue
        rk = r if ranks is None else min(int(ranks[i]), r)
        s = 1.0 if scales is None else float(scales[i])
        A, B = a[i, :rk].astype(np.float64), b[i, :, :rk].astype(np.float64)
        v = A @ xv[t]
        ref = start[t] + s * (B @ v)
        mag = np.abs(start[t]) + s * (np.abs(B) @ (np.abs(A) @ np.abs(xv[t])))
        tol = (k + r + 4) * 2.0 ** -23 * mag
        if rk:
            tol = tol + 2.0 ** -38 * s * np.abs(B).sum(1) * np.abs(v).max()
        assert (np.abs(got[t] - ref) <= tol).all(), t


def test_lora_without_order_and_with_bad_rows():
    """Positions as rows; an order that names rows outside stays inside."""
    rng = np.random.default_rng(4)
    rows, r, n, k = 6, 8, 32, 64
    x = rng.standard_normal((rows, k)).astype(np.float32)
    a = rng.standard_normal((2, r, k)).astype(np.float16)
    b = rng.standard_normal((2, n, r)).astype(np.float16)
    off = torch.tensor([1, 3, 5], dtype=torch.int32, device="cuda")
    xd, ad, bd = (torch.from_numpy(t).cuda() for t in (x, a, b))
    ws = torch.empty(q4k.q4k_lora_ws(rows, r), dtype=torch.uint8, device="cuda")
    for order, named in ((None, {1: (0, 1), 2: (0, 2), 3: (1, 3), 4: (1, 4)}),
                         ([0, 5, -1, 6, 0, 3], {1: (0, 5), 4: (1, 0)})):
        y = torch.full((rows, n), 2.0, device="cuda")
        od = None if order is None else torch.tensor(order, dtype=torch.int32, device="cuda")
        q4k.q4k_lora(xd, ad, bd, y, off, od, n, k, r, 2, rows, ws=ws)
        want = np.full((rows, n), 2.0)
        for _, (i, t) in named.items():
            want[t] = b[i].astype(np.float64) @ (a[i].astype(np.float64) @ x[t].astype(np.float64))
        np.testing.assert_allclose(y.cpu().numpy(), want, rtol=0, atol=1e-3)


def test_lora_non_finite_rows_stay_apart():
    rng = np.random.default_rng(5)
    rows, r, n, k = 5, 4, 16, 32
    x = rng.standard_normal((rows, k)).astype(np.float32)
    x[2, 3] = np.inf
    a = rng.standard_normal((1, r, k)).astype(np.float16)
    b = rng.standard_normal((1, n, r)).astype(np.float16)
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    ws = torch.empty(q4k.q4k_lora_ws(rows, r), dtype=torch.uint8, device="cuda")
    y = torch.empty((rows, n), device="cuda")
    q4k.q4k_lora(torch.from_numpy(x).cuda(), torch.from_numpy(a).cuda(), torch.from_numpy(b).cuda(),
                 y, off, None, n, k, r, 1, rows, ws=ws)
    got = y.cpu().numpy()
    assert not np.isfinite(got[2]).any() and np.isfinite(got[[0, 1, 3, 4]]).all()
