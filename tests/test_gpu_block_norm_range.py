"""GPU tests of q4k_block_norm over the range of f32: rows and factors whose
intermediate products pass it although their results do not.

Where a result is known without a rounding it is compared for equality; the bounds
elsewhere are the documented ones, derived in test_gpu_block_norm.py.
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
