"""GPU parity of the routing (q4k_moe_route), the grouping (q4k_moe_group) and
the combination (q4k_moe_combine) against numpy.

Ids, offsets and orders are whole numbers: equal.  A weight is exp of a
difference of at most one rounding (2^-24 of a difference below 200), an exp
within two steps, a sum of E positive terms and a quotient: within
(E + 8) 2^-24 of itself relative, plus 200 * 2^-24 for the argument.  The
combination sums topk + 1 products in f32: (topk + 2) 2^-24 of the sum of
magnitudes.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from block_quantized_decode_q4_amd import q4k  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    q4k.load_library()
    yield


def _ref_route(logits, topk, renorm):
    m, E = logits.shape
    ids = np.full((m, topk), -1, np.int32)
    weights = np.zeros((m, topk))
    for t in range(m):
        l = logits[t].astype(np.float64)
        l = np.where(np.isnan(l), -np.inf, l)
        order = np.argsort(-l, kind="stable")
        chosen = [e for e in order[:topk] if l[e] > -np.inf]
        if not chosen:
            continue
        top = l[chosen[0]]
        with np.errstate(invalid="ignore"):           # inf - inf, replaced by 1
            p = np.where(l == -np.inf, 0.0, np.where(l == top, 1.0, np.exp(l - top)))
        total = p[chosen].sum() if renorm else p.sum()
        ids[t, :len(chosen)] = chosen
        weights[t, :len(chosen)] = p[chosen] / total
    return ids, weights


def _ref_group(flat, groups):
    inside = (flat >= 0) & (flat < groups)
    key = np.where(inside, flat, groups)
    order = np.argsort(key, kind="stable").astype(np.int32)
    order[inside.sum():] = -1
    offsets = np.searchsorted(np.sort(key), np.arange(groups + 1), side="left").astype(np.int32)
    return offsets, order


def _ws(slots, groups, topk):
    n = q4k.q4k_moe_group_ws(slots, groups, topk)
    return torch.empty(n, dtype=torch.uint8, device="cuda") if n else None


def _route(logits, E, topk, m, renorm, stride=0, group=True):
    ids = torch.full((m, topk), 77, dtype=torch.int32, device="cuda")
    weights = torch.full((m, topk), float("nan"), device="cuda")
    off = torch.full((E + 1,), 99, dtype=torch.int32, device="cuda") if group else None
    order = torch.full((m * topk,), 99, dtype=torch.int32, device="cuda") if group else None
    q4k.q4k_moe_route(logits, ids, weights, E, topk, m, renorm=renorm, offsets=off, order=order,
                      ws=_ws(m * topk, E, topk) if group else None, logits_stride=stride)
    torch.cuda.synchronize()
    return ids, weights, off, order


CASES = [(1, 1, 1), (1, 4, 2), (1, 64, 8), (8, 64, 8), (3, 65, 3), (64, 8, 2), (65, 8, 8),
         (100, 128, 8), (513, 5, 1), (300, 100, 7), (2000, 60, 6), (1000, 1024, 32),
         (4097, 256, 8), (700, 512, 1), (16, 32, 32), (17, 32, 32), (1, 1024, 32),
         (24, 64, 8), (25, 64, 8), (128, 9, 1), (129, 9, 1), (16, 300, 4), (17, 300, 4)]


@pytest.mark.parametrize("m,E,topk", CASES)
@pytest.mark.parametrize("renorm", [True, False])
def test_route(m, E, topk, renorm):
    rng = np.random.default_rng(m * 131 + E + topk)
    logits = (rng.standard_normal((m, E)) * 3).astype(np.float32)
    # ties everywhere in some rows, masks, rows with nothing left
    logits[::3] = np.round(logits[::3])
    if m > 2:
        logits[1, : E // 2] = -np.inf
        logits[2] = -np.inf
        logits[2, E // 2] = np.nan
    if m > 8:
        logits[5] = -np.inf
        logits[5, E - 1] = 2.0
        logits[6] = 0.0
        logits[6, ::2] = -0.0
        logits[7, E // 3] = np.inf
    print("route m=%d E=%d topk=%d renorm=%s" % (m, E, topk, renorm), flush=True)
    ids, weights, off, order = _route(torch.from_numpy(logits).cuda(), E, topk, m, renorm)
    ids_ref, w_ref = _ref_route(logits, topk, renorm)
    assert np.array_equal(ids.cpu().numpy(), ids_ref)
    err = np.abs(weights.cpu().numpy() - w_ref)
    assert (err <= (E + 208) * 2.0 ** -24 * w_ref + 2.0 ** -149).all()
    off_ref, order_ref = _ref_group(ids_ref.reshape(-1), E)
    assert np.array_equal(off.cpu().numpy(), off_ref)
    assert np.array_equal(order.cpu().numpy(), order_ref)


def test_route_without_grouping_and_with_strided_logits():
    rng = np.random.default_rng(3)
    for m in (5, 900):
        logits = rng.standard_normal((m, 72)).astype(np.float32)
        full = torch.from_numpy(logits).cuda()
        ids, weights, _, _ = _route(full, 40, 4, m, True, stride=72, group=False)
        ids_ref, w_ref = _ref_route(logits[:, :40], 4, True)
        assert np.array_equal(ids.cpu().numpy(), ids_ref)
        ids2, weights2, off, order = _route(full, 40, 4, m, True, stride=72)
        assert torch.equal(ids, ids2) and torch.equal(weights, weights2)


@pytest.mark.parametrize("count,groups", [(1, 1), (5, 3), (512, 1024), (513, 1024), (513, 1),
                                          (5000, 7), (70001, 33), (200000, 1000)])
def test_group(count, groups):
    rng = np.random.default_rng(count + groups)
    ids = rng.integers(-2, groups + 2, size=count).astype(np.int32)
    ids[: count // 2] = np.minimum(ids[: count // 2], groups // 2)     # a crowded half
    ids[0] = 2 ** 31 - 1
    print("group count=%d groups=%d" % (count, groups), flush=True)
    off = torch.full((groups + 1,), 99, dtype=torch.int32, device="cuda")
    order = torch.full((count,), 99, dtype=torch.int32, device="cuda")
    q4k.q4k_moe_group(torch.from_numpy(ids).cuda(), off, order, count, groups,
                      ws=_ws(count, groups, 1))
    off_ref, order_ref = _ref_group(ids, groups)
    assert np.array_equal(off.cpu().numpy(), off_ref)
    assert np.array_equal(order.cpu().numpy(), order_ref)


def test_group_all_in_one_and_none():
    for ids_value, groups in ((3, 5), (-1, 5)):
        for count in (100, 3000):
            ids = torch.full((count,), ids_value, dtype=torch.int32, device="cuda")
            off = torch.empty(groups + 1, dtype=torch.int32, device="cuda")
            order = torch.empty(count, dtype=torch.int32, device="cuda")
            q4k.q4k_moe_group(ids, off, order, count, groups, ws=_ws(count, groups, 1))
            off_ref, order_ref = _ref_group(ids.cpu().numpy(), groups)
            assert np.array_equal(off.cpu().numpy(), off_ref)
            assert np.array_equal(order.cpu().numpy(), order_ref)


@pytest.mark.parametrize("m,n,topk,residual,masked", [
    (1, 1, 1, False, False), (1, 2048, 8, True, False), (3, 1027, 2, True, True),
    (5, 4096, 32, False, True), (700, 260, 3, True, True), (2, 33, 5, False, True),
    (9, 2, 2, True, False), (9, 3, 1, True, True), (9, 5, 4, True, True), (40, 1023, 2, True, False),
    (300, 1025, 3, True, True), (70, 7, 8, True, True)])
def test_combine(m, n, topk, residual, masked):
    rng = np.random.default_rng(m + n)
    y = rng.standard_normal((m * topk, n)).astype(np.float32)
    w = rng.random((m, topk)).astype(np.float32)
    ids = rng.integers(0, 9, size=(m, topk)).astype(np.int32)
    if masked:
        ids[rng.random((m, topk)) < 0.4] = -1
        ids[0] = -1                                   # nothing left: the residual, or 0
        y[ids.reshape(-1) < 0] = np.nan               # never written, never read
    r = rng.standard_normal((m, n)).astype(np.float32) if residual else None
    print("combine m=%d n=%d topk=%d" % (m, n, topk), flush=True)
    out = torch.full((m, n), float("nan"), device="cuda")
    r_d = torch.from_numpy(r).cuda() if residual else None
    y_d, w_d, ids_d = (torch.from_numpy(a).cuda() for a in (y, w, ids))
    q4k.q4k_moe_combine(y_d, w_d, ids_d, out, n, topk, m, residual=r_d)
    keep = (ids >= 0)[:, :, None]
    terms = np.where(keep, w[:, :, None].astype(np.float64) * np.nan_to_num(y).reshape(m, topk, n), 0)
    ref = terms.sum(1) + (0 if r is None else r)
    mag = np.abs(terms).sum(1) + (0 if r is None else np.abs(r))
    got = out.cpu().numpy()
    assert (np.abs(got - ref) <= (topk + 2) * 2.0 ** -24 * mag).all()
    if residual:                                       # in place
        q4k.q4k_moe_combine(y_d, w_d, ids_d, r_d, n, topk, m, residual=r_d)
        assert torch.equal(r_d, out)
    if not masked:
        q4k.q4k_moe_combine(y_d, w_d, None, out, n, topk, m, residual=None)
        assert (np.abs(out.cpu().numpy() - terms.sum(1)) <= (topk + 2) * 2.0 ** -24 * mag).all()


def test_route_takes_views_of_wider_rows():
    g = torch.Generator().manual_seed(72)
    wide = torch.randn((9, 80), generator=g).cuda()
    a = _route(wide[:, :64], 64, 4, 9, True, stride=80)
    b = _route(wide[:, :64].contiguous(), 64, 4, 9, True)
    for u, v in zip(a, b):
        assert torch.equal(u, v)
    with pytest.raises(ValueError):
        _route(wide[:, :64], 64, 4, 9, True, stride=96)
    with pytest.raises(ValueError):
        _route(wide[:, :64], 64, 4, 9, True)
    with pytest.raises(ValueError):
        _route(wide[:, :64], 64, 4, 10, True, stride=80)


def test_group_refuses_a_workspace_said_to_be_longer():
    n = 20000
    ids = torch.zeros(n, dtype=torch.int32, device="cuda")
    off = torch.empty(5, dtype=torch.int32, device="cuda")
    order = torch.empty(n, dtype=torch.int32, device="cuda")
    ws = torch.empty(16, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError):
        q4k.q4k_moe_group(ids, off, order, n, 4, ws=ws, ws_bytes=1 << 20)
    with pytest.raises(q4k.Q4KError):
        q4k.q4k_moe_group(ids, off, order, n, 4, ws=ws)
