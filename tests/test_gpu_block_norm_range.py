"""GPU tests of q4k_block_norm over the range of f32: rows and factors whose
intermediate products pass it although their results do not.

Where a result is known without a rounding it is compared for equality; the bounds
elsewhere are derived at each test or in test_gpu_block_norm.py.
"""
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


def _rand(g, *shape):
    return torch.randn(shape, device="cuda", generator=g)


CONSTANTS = (0.0, 1e-30, 5.0, 1e30, -7e35, 1e37, -1e38, 3.4028234663852886e38)


@pytest.mark.parametrize("k", [1, 7, 512, 2049, 8200, 40000])
@pytest.mark.parametrize("eps", [1e-5, 1e-30, 1e-45])
def test_layer_norm_of_constant_rows(k, eps):
    """Every element is its row's mean, so a normed row is 0 whatever its size: y is
    the bias, through the norm of x (as h) and the one of h."""
    g = torch.Generator(device="cuda").manual_seed(k)
    m = len(CONSTANTS)
    x = torch.tensor(CONSTANTS, device="cuda")[:, None].expand(m, k).contiguous()
    w, b = _rand(g, k), _rand(g, k)
    h, y = torch.empty((m, k), device="cuda"), torch.empty((m, k), device="cuda")
    print("constant rows", k, eps, flush=True)
    q4k.q4k_block_norm(x, w, k, m, kind=q4k.Q4K_NORM_LAYER, bias=b, y=y, eps=eps)
    assert torch.equal(y, b.expand(m, k))
    q4k.q4k_block_norm(x, w, k, m, kind=q4k.Q4K_NORM_LAYER, y=y, eps=eps)
    assert bool((y == 0).all())
    q4k.q4k_block_norm(x, None, k, m, kind=q4k.Q4K_NORM_LAYER, post_weight=w, post_bias=b,
                       sum_out=h, eps=eps)
    assert torch.equal(h, b.expand(m, k))


# gate, scale, x: gate x passes f32 and scale gate x does not; scale gate does and scale
# gate x does not
FACTORS = [(10.0, 0.01, 1e38), (-3e30, 1e-30, 2e20), (1e30, 1e20, 1e-30), (3e38, 3e38, 1e-45)]


@pytest.mark.parametrize("gate,scale,x", FACTORS)
@pytest.mark.parametrize("m,k", [(1, 9), (2, 64), (300, 4100), (2, 20000)])
def test_gate_and_scale_far_from_one(gate, scale, x, m, k):
    """Without a norm of x, h is off by the rounding of gate x (half a step, 2^-24, of
    it) and its own."""
    g = torch.Generator(device="cuda").manual_seed(k)
    xs = x * (1 + torch.rand((m, k), device="cuda", generator=g))
    gates = gate * (1 + 0.1 * torch.rand((m, k), device="cuda", generator=g))
    scale = torch.tensor(scale).item()
    res = (xs.double() * gates.double() * scale * _rand(g, m, k).double()).float()
    print("factors", gate, scale, x, m, k, flush=True)
    for r in (None, res):
        for rows in (1, m):
            f = gates[:rows].contiguous()
            h = torch.full((m, k), float("nan"), device="cuda")
            q4k.q4k_block_norm(xs, None, k, m, gate=f, gate_stride=0 if rows == 1 else k,
                               scale=scale, residual=r, sum_out=h)
            part = xs.double() * f.double() * scale
            ref = part if r is None else part + r.double()
            err = 2.0 ** -24 * (1 + 2.0 ** -20) * (ref.abs() + part.abs())
            assert bool(((h.double() - ref).abs() <= err).all())
            if r is not None:                  # in place
                q4k.q4k_block_norm(xs, None, k, m, gate=f, gate_stride=0 if rows == 1 else k,
                                   scale=scale, residual=(over := r.clone()), sum_out=over)
                assert torch.equal(over, h)


def test_a_norm_past_f32_that_comes_back():
    """The normed value times post_weight passes f32; with post_bias, or through the
    gate, h does not."""
    k = 64
    x = torch.ones((1, k), device="cuda")
    x[0, 1::2] = -1
    x[0, 0] = 4                                # its norm is about 3.6
    w = torch.full((k,), 1.5e38, device="cuda")
    b = torch.zeros(k, device="cuda")
    b[0] = -3e38
    v = x.double()
    part = v / v.square().mean().sqrt() * w.double()
    assert bool(part[0, 0] > 3.5e38)
    h = torch.empty((1, k), device="cuda")
    for bias, gate, scale in ((b, None, 1.0), (None, 0.125, 1.0), (None, None, 0.125),
                              (b, 3.0, 0.25), (None, 0.0, 1.0)):
        gates = None if gate is None else torch.full((k,), gate, device="cuda")
        q4k.q4k_block_norm(x, None, k, 1, post_weight=w, post_bias=bias, gate=gates, scale=scale,
                           sum_out=h, eps=0.0)
        f = scale * (1.0 if gate is None else gate)
        beside = torch.zeros_like(part) if bias is None else bias.double()
        ref = (part + beside) * f
        assert bool((ref.abs() < 3.4e38).all())
        err = 2.0 ** -21 * abs(f) * (part.abs() + beside.abs())
        assert bool(((h.double() - ref).abs() <= err).all())
