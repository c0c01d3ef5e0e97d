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
