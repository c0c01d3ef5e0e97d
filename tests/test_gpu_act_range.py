"""GPU test of the activations' documented bound (include/q4k.h) where the exponential
overflows and the values vanish: nothing is added to it, but for large z > 0, where
act is z, 0 or 1 to a rounding, 2^-22 of the value is held instead where that is less.
"""
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


def _values():
    """z of both signs: steps through the ranges where e^z leaves f32 and the results
    fall below 2^-100, 2^-126 and 2^-149, and all sizes."""
    steps = torch.cat([torch.linspace(0, 64, 2048), torch.linspace(64, 112, 4096),
                       torch.linspace(3, 15, 1024), torch.logspace(-37.9, 38.5, 1024)])
    return torch.cat([-steps, steps]).cuda()


@pytest.mark.parametrize("act", B.ACTS)
@pytest.mark.parametrize("product", ["q4", "f16"])
def test_documented_bound(act, product):
    """Products whose sums are 0 and whose z is the bias."""
    z = _values()
    n, k = z.numel(), 256
    x = torch.zeros((1, k), device="cuda")
    y = torch.full((1, n), float("nan"), device="cuda")
    if product == "q4":
        w = torch.zeros((n, 144), device="cuda", dtype=torch.uint8)
        q4k.q4k_gemv_act(w, x, y, n, k, 1, act=act, bias=z)
    else:
        w = torch.zeros((n, k), device="cuda", dtype=torch.float16)
        q4k.q4k_f16_gemm_act(w, x.half(), y, 1, n, k, act=act, bias=z)
    z = z.double()[None]
    ref = B.act64(z, act)
    err = B.act_error(z, act)
    assert bool(ref.isfinite().all()) and bool(err.isfinite().all())
    err = torch.where(z > 64, torch.minimum(err, 2.0 ** -22 * ref.abs()), err)
    B.assert_within(y, ref, err, "act %d" % act)
