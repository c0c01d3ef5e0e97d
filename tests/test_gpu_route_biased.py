"""GPU parity of the routing by biased scores (q4k_moe_route_biased) against the
definition in numpy f64.

Ids, offsets and orders are whole numbers: equal (scores within 1e-12 of one
another, but for equal ones, are not among the inputs).  Weights are f64 rounded
once: 2^-24 of themselves, and 1e-13 for the exps' and sums' roundings.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import block_ops as B  # noqa: E402
from block_quantized_decode_q4_amd import q4k  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    q4k.load_library()
    yield


def _ref_group(flat, groups):
    inside = (flat >= 0) & (flat < groups)
    key = np.where(inside, flat, groups)
    order = np.argsort(key, kind="stable").astype(np.int32)
    order[inside.sum():] = -1
    offsets = np.searchsorted(np.sort(key), np.arange(groups + 1), side="left").astype(np.int32)
    return offsets, order


def _run(logits, bias, sigmoid, parts, keep, topk, renorm, scale, stride=0, group=True):
    m = logits.shape[0]
    E = logits.shape[1] if bias is None else bias.numel()
    ids = torch.full((m, topk), 77, dtype=torch.int32, device="cuda")
    weights = torch.full((m, topk), float("nan"), device="cuda")
    off = torch.full((E + 1,), 99, dtype=torch.int32, device="cuda") if group else None
    order = torch.full((m * topk,), 99, dtype=torch.int32, device="cuda") if group else None
    nb = q4k.q4k_moe_group_ws(m * topk, E, topk)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda") if group and nb else None
    q4k.q4k_moe_route_biased(
        logits, ids, weights, E, topk, m, bias=bias,
        score=q4k.Q4K_SCORE_SIGMOID if sigmoid else q4k.Q4K_SCORE_SOFTMAX, groups=parts,
        topk_groups=keep, renorm=renorm, scale=scale, offsets=off, order=order, ws=ws,
        logits_stride=stride)
    torch.cuda.synchronize()
    return [None if t is None else t.cpu().numpy() for t in (ids, weights, off, order)]


def _check(logits, bias, sigmoid, parts, keep, topk, renorm, scale):
    got = _run(torch.from_numpy(logits).cuda(),
               None if bias is None else torch.from_numpy(bias).cuda(), sigmoid, parts, keep, topk,
               renorm, scale)
    ids, weights = B.route64(logits, bias, sigmoid, parts, keep, topk, renorm, scale)
    assert np.array_equal(got[0], ids)
    err = np.abs(got[1] - weights)
    assert (err <= (2.0 ** -24 + 1e-13) * np.abs(weights) + 2.0 ** -149).all()
    off, order = _ref_group(ids.reshape(-1), logits.shape[1])
    assert np.array_equal(got[2], off) and np.array_equal(got[3], order)


# tokens, experts, topk, groups, groups that stay
CASES = [(1, 1, 1, 1, 1), (1, 4, 2, 2, 1), (2, 64, 6, 1, 1), (16, 64, 8, 8, 4), (3, 65, 3, 5, 2),
         (64, 8, 2, 8, 3), (100, 128, 8, 4, 2), (513, 6, 1, 3, 1), (300, 100, 7, 10, 9),
         (1000, 256, 8, 8, 4), (700, 512, 4, 16, 5), (40, 1024, 32, 64, 20), (16, 320, 5, 64, 1),
         (33, 32, 32, 1, 1), (9, 48, 16, 3, 1), (2000, 60, 6, 6, 6), (5, 256, 8, 2, 1),
         (31, 192, 8, 64, 64), (257, 160, 6, 8, 3), (60, 24, 3, 24, 11)]


@pytest.mark.parametrize("m,E,topk,parts,keep", CASES)
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_route(m, E, topk, parts, keep, sigmoid, renorm):
    rng = np.random.default_rng(m * 131 + E + topk)
    logits = (rng.standard_normal((m, E)) * 2).astype(np.float32)
    bias = (rng.standard_normal(E) * (0.2 if sigmoid else 0.5 / E)).astype(np.float32)
    logits[::3] = np.round(logits[::3])        # ties wherever the biases are alike
    bias[::2] = bias[0]
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
        logits[8] = -300.0                     # a sigmoid that f32 loses, f64 keeps
    print("route", m, E, topk, parts, keep, sigmoid, renorm, flush=True)
    for b in (bias, None):
        _check(logits, b, sigmoid, parts, keep, topk, renorm, 2.5 if renorm else 1.0)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_biases_that_are_not_finite(sigmoid):
    """-infinity and NaN keep an expert out, +infinity puts it first, and an
    expert that is kept out still counts in a softmax's sum."""
    rng = np.random.default_rng(4)
    logits = rng.standard_normal((50, 32)).astype(np.float32)
    bias = np.zeros(32, np.float32)
    bias[[1, 2, 3]] = -np.inf
    bias[9] = np.nan
    bias[[20, 30]] = np.inf
    for parts, keep in ((1, 1), (8, 2)):
        for renorm in (False, True):
            _check(logits, bias, sigmoid, parts, keep, 6, renorm, 1.0)
    bias[:] = -np.inf                          # nobody to choose
    _check(logits, bias, sigmoid, 4, 2, 6, True, 1.0)
    bias[5] = 0
    _check(logits, bias, sigmoid, 4, 2, 6, True, 1.0)


def test_scores_closer_than_f32():
    """Choices that only f64 tells apart: scores a fraction of a step of f32 from one another."""
    m, E = 64, 64
    rng = np.random.default_rng(5)
    step = np.float32(2.0 ** -21)
    logits = np.zeros((m, E), np.float32)
    for t in range(m):
        logits[t] = np.float32(5.0) + step * rng.permutation(E).astype(np.float32)
    bias = np.zeros(E, np.float32)
    # sigmoid at 5 has slope 0.0066: neighbours are 3.2e-9 apart, a 19th of f32's step
    for parts, keep in ((1, 1), (8, 3)):
        _check(logits, bias, True, parts, keep, 8, True, 1.0)
        _check(logits, bias, False, parts, keep, 8, True, 1.0)


def test_a_sum_of_zero():
    """Scores that vanish in f64 too give weights 0, not NaN."""
    logits = np.full((3, 8), -1000.0, np.float32)
    _check(logits, np.arange(8, dtype=np.float32), True, 1, 1, 2, True, 1.0)


@pytest.mark.parametrize("m", [5, 900])
def test_strided_logits_without_grouping(m):
    E, topk = 96, 4
    g = torch.Generator(device="cuda").manual_seed(m)
    wide = torch.full((m, E + 5), float("nan"), device="cuda")
    wide[:, :E] = torch.randn((m, E), device="cuda", generator=g)
    bias = torch.randn(E, device="cuda", generator=g) * 0.1
    ids, weights, _, _ = _run(wide, bias, True, 4, 2, topk, True, 1.0, stride=E + 5, group=False)
    ref = B.route64(wide[:, :E].cpu().numpy(), bias.cpu().numpy(), True, 4, 2, topk, True, 1.0)
    assert np.array_equal(ids, ref[0])
    assert (np.abs(weights - ref[1]) <= (2.0 ** -24 + 1e-13) * ref[1]).all()


def test_without_a_bias_as_the_plain_routing():
    """Softmax scores without bias and groups choose what q4k_moe_route chooses."""
    m, E, topk = 300, 100, 7
    g = torch.Generator(device="cuda").manual_seed(7)
    logits = torch.randn((m, E), device="cuda", generator=g)
    ids, weights, off, order = _run(logits, None, False, 1, 1, topk, True, 1.0)
    i2 = torch.empty((m, topk), dtype=torch.int32, device="cuda")
    w2 = torch.empty((m, topk), device="cuda")
    q4k.q4k_moe_route(logits, i2, w2, E, topk, m)
    assert np.array_equal(ids, i2.cpu().numpy())
    assert np.abs(weights - w2.cpu().numpy()).max() < 1e-5
