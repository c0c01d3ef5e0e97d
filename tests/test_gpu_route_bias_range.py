"""GPU parity of q4k_moe_route_biased with biases over the range of f32, against the
definition in numpy f64: ids, offsets and orders equal, weights within the bounds of
test_gpu_route_biased.py.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from block_quantized_decode_q4_amd import q4k  # noqa: E402
from test_gpu_route_biased import _check  # noqa: E402

pytestmark = pytest.mark.gpu

LOWEST = np.finfo(np.float32).min


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    q4k.load_library()
    yield


def _logits(rng, m, E):
    logits = (rng.standard_normal((m, E)) * 2).astype(np.float32)
    logits[::3] = np.round(logits[::3])        # equal scores
    return logits


# tokens, experts, topk, groups, groups that stay
GROUPED = [(1, 8, 2, 4, 2), (5, 64, 6, 8, 4), (40, 256, 8, 8, 4), (300, 96, 4, 32, 9),
           (12, 512, 8, 4, 2), (33, 1024, 9, 64, 20), (7, 24, 3, 24, 11)]


@pytest.mark.parametrize("m,E,topk,parts,keep", GROUPED)
@pytest.mark.parametrize("sigmoid", [False, True])
def test_groups_whose_values_pass_f32(m, E, topk, parts, keep, sigmoid):
    """Two biases whose sum passes f32 either way: the group's value is their sum all
    the same."""
    rng = np.random.default_rng(E + parts)
    logits = _logits(rng, m, E)
    each = E // parts
    group = np.arange(E) // each
    for name, bias in (
            ("all lowest", np.full(E, LOWEST)),
            ("two groups of others", np.where(group % (parts // 2 + 1) == 1, 0.0, LOWEST)),
            ("near the lowest", LOWEST * (1 - 0.4 * rng.random(E))),
            ("near the largest", -LOWEST * (1 - 0.4 * rng.random(E))),
            ("steps of the lowest", LOWEST * (1 - np.arange(E) % 3 * 2.0 ** -23))):
        bias = bias.astype(np.float32)
        bias[E // 2] = np.nan                  # a group with an expert kept out
        print("values", name, m, E, topk, parts, keep, sigmoid, flush=True)
        _check(logits, bias, sigmoid, parts, keep, topk, True, 1.0)


CHOICES = [(16, 64, 6, 1, 1), (9, 200, 8, 1, 1), (600, 64, 8, 8, 4), (900, 256, 8, 8, 4),
           (40, 512, 6, 16, 5), (6, 1024, 32, 1, 1), (50, 48, 5, 24, 7)]


@pytest.mark.parametrize("m,E,topk,parts,keep", CHOICES)
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_far_biases_among_others(m, E, topk, parts, keep, sigmoid, renorm):
    """Experts far out of the others' range, either way: they are chosen first or last
    and the others' order is that of their own values."""
    rng = np.random.default_rng(E + topk)
    logits = _logits(rng, m, E)
    scale = 0.2 if sigmoid else 0.5 / E
    near = (rng.standard_normal(E) * scale).astype(np.float32)
    near[::2] = near[0]                        # equal values among them
    at = rng.permutation(E)
    for far in (-1e9, -1e30, LOWEST, 1e6, 1e30, -LOWEST, np.inf, -np.inf):
        for count in (1, 3, E // 2):
            bias = near.copy()
            bias[at[:count]] = far
            print("far", far, count, m, E, topk, parts, keep, sigmoid, renorm, flush=True)
            _check(logits, bias, sigmoid, parts, keep, topk, renorm, 1.5)
    bias = near.copy()                         # several sizes at once
    bias[at[:6]] = [-1e9, 1e6, -300.0, 2e3, -LOWEST, LOWEST]
    _check(logits, bias, sigmoid, parts, keep, topk, renorm, 1.5)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_groups_that_meet_in_their_sums(sigmoid):
    """Groups whose largest values are far apart and whose sums are near: a value off by
    its own size's rounding, not by the others'."""
    rng = np.random.default_rng(11)
    E, parts = 64, 8
    logits = _logits(rng, 30, E)
    bias = (rng.standard_normal(E) * 0.1).astype(np.float32) - 50
    for p in range(parts):                     # sums of 1 and a little, from summands of all sizes
        size = np.float32(4.0 ** p)
        bias[8 * p + 1] = size
        bias[8 * p + 5] = np.float32(1 + rng.random() * 2.0 ** -20) - size
    for keep in range(1, parts + 1):
        _check(logits, bias, sigmoid, parts, keep, min(6, 8 * keep), True, 1.0)
    logits[:, :] = 0.25                        # and the scores the same
    for keep in range(1, parts + 1):
        _check(logits, bias, sigmoid, parts, keep, min(6, 8 * keep), True, 1.0)


@pytest.mark.parametrize("E,parts,keep", [(64, 1, 1), (64, 8, 3), (256, 1, 1), (256, 8, 4),
                                          (512, 16, 5), (1024, 1, 1), (1024, 64, 9)])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_values_that_meet_through_their_biases(E, parts, keep, sigmoid):
    """Biases that take every score to the same value but for the biases' own rounding,
    1e-8 of it: an error that f32's scores have in common, of the sum of all, counts
    in each by its score's size."""
    rng = np.random.default_rng(E + parts)
    for spread in (0.5, 2.0, 6.0):
        logits = (rng.standard_normal((1, E)) * spread).astype(np.float32)
        logits[0, 0] = 5.5 if spread == 0.5 else 3 * spread
        l = logits[0].astype(np.float64)
        s = 1 / (1 + np.exp(-l)) if sigmoid else np.exp(l - l.max()) / np.exp(l - l.max()).sum()
        bias = (s.max() - s).astype(np.float32)
        _check(logits, bias, sigmoid, parts, keep, 8, True, 1.0)
        _check(np.repeat(logits, 400, 0), bias, sigmoid, parts, keep, 8, False, 1.0)
