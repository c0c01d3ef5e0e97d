"""GPU test of the bounds that include/q4k.h gives for q4k_block_norm, with nothing
added to them.

Half steps of f32 (2^-24): a normed value carries the factor r's rounding, its
difference from the mean (the product exact, two steps), the product with r and the
one with the weight, five; the bias's addition is the sixth (y: together with the
weight's product), the gate's product the seventh, the residual's addition the
eighth, where the residual has its own term.  A layer norm's mean is two f32 numbers,
2^-49 of it off, and the f64 sum's share (exact where the mean is far from 0, whose
elements are of one size) below another 2^-49: 2^-48 m, m the mean in units of the
deviation.  The reference's own f64 sums are off by a few 2^-53 m, a thirtieth of
that.
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


def _rand(g, *shape):
    return torch.randn(shape, device="cuda", generator=g)


def _far(v, layer, weight, eps):
    """The term of a layer norm whose mean is far from 0."""
    if not layer:
        return 0.0
    mean = v.mean(1, keepdim=True)
    deviation = torch.sqrt((v - mean).square().mean(1, keepdim=True) + eps)
    return 2.0 ** -48 * (mean / deviation).abs() * weight.double().abs()


MEANS = (0.0, 1.0, -300.0, 2e5)


@pytest.mark.parametrize("m,k", [(4, 100), (8, 2049), (4, 4096), (4, 8200), (4, 40000),
                                 (1100, 8208), (300, 4096)])
@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("x_type", [torch.float32, torch.float16, torch.bfloat16])
def test_documented_bounds(m, k, layer, x_type):
    g = torch.Generator(device="cuda").manual_seed(k + m)
    eps, scale = 1e-5, torch.tensor(-0.22).item()
    far = torch.tensor(MEANS, device="cuda").repeat((m + 3) // 4)[:m, None]
    if x_type is torch.float16:
        far = far.clamp(max=3e4)
    x = (_rand(g, m, k) * (1 + far.abs() / 100) + far).to(x_type)
    if m >= 8:                                 # deviations of a few steps around the mean
        x[3::4] = (x[3::4].double() * 2.0 ** -9 + 2e4).to(x_type)
    pw, w, gate = _rand(g, k), _rand(g, k), _rand(g, m, k)
    kind = q4k.Q4K_NORM_LAYER if layer else q4k.Q4K_NORM_RMS
    print("bounds", m, k, layer, x_type, flush=True)
    for pb, b, res in ((None, None, None), (_rand(g, k), _rand(g, k), _rand(g, m, k) * 100)):
        h = torch.full((m, k), float("nan"), device="cuda")
        y = torch.full((m, k), float("nan"), device="cuda")
        q4k.q4k_block_norm(x, w, k, m, kind=kind, post_weight=pw, post_bias=pb, gate=gate,
                           gate_stride=k, scale=scale, residual=res, bias=b, sum_out=h, y=y,
                           eps=eps)
        f = scale * gate.double()
        part = B.norm64(x.double(), layer, pw, None, eps)
        beside = torch.zeros_like(part) if pb is None else pb.double()
        r = torch.zeros_like(part) if res is None else res.double()
        err = 2.0 ** -21 * f.abs() * (part.abs() + beside.abs()) + 2.0 ** -24 * r.abs()
        err = err + f.abs() * _far(x.double(), layer, pw, eps)
        err = err + 2.0 ** -146 * (abs(scale) + f.abs())
        B.assert_within(h, (part + beside) * f + r, err, "h")
        part = B.norm64(h.double(), layer, w, None, eps)
        beside = torch.zeros_like(part) if b is None else b.double()
        err = 6 * 2.0 ** -24 * (part.abs() + beside.abs()) + _far(h.double(), layer, w, eps)
        B.assert_within(y, part + beside, err, "y")
