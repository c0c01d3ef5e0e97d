"""Grouping and routing at the limits of their one-workgroup forms, and routing
among logits of which several are +infinite.  References and bounds are those
of test_gpu_moe.py."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from block_quantized_decode_q4_amd import q4k  # noqa: E402
from test_gpu_moe import _ref_group, _ref_route, _route, _ws  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    q4k.load_library()
    yield


@pytest.mark.parametrize("count", [1, 2, 3, 127, 128, 129, 189, 190, 191, 192, 193, 194, 255, 257])
@pytest.mark.parametrize("groups", [1, 7, 64, 1024])
def test_group_near_the_one_workgroup_limit(count, groups):
    rng = np.random.default_rng(count * 1031 + groups)
    ids = rng.integers(-2, groups + 2, size=count).astype(np.int32)
    ids[: count // 3] = groups - 1
    ids[-1] = groups - 1 if count % 2 else -2 ** 31
    print("group count=%d groups=%d" % (count, groups), flush=True)
    off = torch.full((groups + 9,), 99, dtype=torch.int32, device="cuda")
    order = torch.full((count + 8,), 99, dtype=torch.int32, device="cuda")
    q4k.q4k_moe_group(torch.from_numpy(ids).cuda(), off, order, count, groups,
                      ws=_ws(count, groups, 1))
    off_ref, order_ref = _ref_group(ids, groups)
    assert np.array_equal(off.cpu().numpy()[: groups + 1], off_ref)
    assert np.array_equal(order.cpu().numpy()[:count], order_ref)
    assert bool((off[groups + 1:] == 99).all()) and bool((order[count:] == 99).all())


# (256 and 257 experts: 16 lanes or a wave a token; 24, 128 and 16 tokens: the most
# that one workgroup takes)
@pytest.mark.parametrize("m,E,topk", [(24, 64, 8), (25, 64, 8), (128, 256, 1), (129, 256, 1), (16, 257, 12),
                                      (17, 257, 12), (6, 1024, 32), (7, 1024, 32), (5, 16, 16)])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_with_several_infinite_logits(m, E, topk, renorm):
    rng = np.random.default_rng(m + E + topk)
    logits = (rng.standard_normal((m, E)) * 3).astype(np.float32)
    for t in range(m):                    # from none to more than topk of them
        logits[t, rng.permutation(E)[: min(t % (topk + 3), E)]] = np.inf
        if t % 4 == 1:
            logits[t, rng.permutation(E)[: E // 2]] = -np.inf
        if t % 4 == 2:
            logits[t, rng.permutation(E)[: E // 2]] = np.nan
    print("route infinities m=%d E=%d topk=%d renorm=%s" % (m, E, topk, renorm), flush=True)
    ids, weights, off, order = _route(torch.from_numpy(logits).cuda(), E, topk, m, renorm)
    ids_ref, w_ref = _ref_route(logits, topk, renorm)
    assert np.array_equal(ids.cpu().numpy(), ids_ref)
    err = np.abs(weights.cpu().numpy() - w_ref)
    assert (err <= (E + 208) * 2.0 ** -24 * w_ref + 2.0 ** -149).all()
    off_ref, order_ref = _ref_group(ids_ref.reshape(-1), E)
    assert np.array_equal(off.cpu().numpy(), off_ref)
    assert np.array_equal(order.cpu().numpy(), order_ref)
