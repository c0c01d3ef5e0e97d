"""GPU test of the Q4_K products with an epilogue for several vectors and so many rows
that a workgroup's sums do not meet in LDS: each goes through the epilogue where it
is formed.  Bit for bit the plain product's sums, then a rounding each of relu (none),
the gate's product and the residual's addition."""
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


# n, k, m and the kernel that the shape must take
SHAPES = [(1790001, 2048, 2, 4), (249999, 512, 9, 5), (1500000, 256, 5, 5), (350001, 256, 23, 6),
          (300003, 768, 32, 6)]


@pytest.mark.parametrize("n,k,m,kernel", SHAPES)
def test_sums_that_do_not_meet_in_lds(n, k, m, kernel):
    plan = q4k.q4k_plan(n, k, m)
    assert plan.kernel == kernel and (k // 256 + 7) // 8 * 8 == plan.cols_per_task
    assert plan.lds_bytes + 8 * m * plan.rows_per_block > 160 * 1024
    g = torch.Generator(device="cuda").manual_seed(m)
    w = B.random_q4k(g, n, k)
    x = torch.randn((m, k), device="cuda", generator=g)
    res = torch.randn((m, n), device="cuda", generator=g)
    y, plain = torch.empty((m, n), device="cuda"), torch.empty((m, n), device="cuda")
    print("sums", n, k, m, kernel, flush=True)
    q4k.q4k_gemv(w, x, plain, n, k, m)
    y16 = torch.empty((m, n), device="cuda", dtype=torch.float16)
    q4k.q4k_gemv_act(w, x, y, n, k, m, act=q4k.Q4K_ACT_RELU, residual=res, y16=y16)
    ref = plain.clamp(min=0) + res
    assert torch.equal(y, ref) and torch.equal(y16, ref.half())
    over = res.clone()                         # y over the residual, and over the gate
    q4k.q4k_gemv_act(w, x, over, n, k, m, act=q4k.Q4K_ACT_RELU, residual=over)
    assert torch.equal(over, ref)
    over = res.clone()
    q4k.q4k_gemv_act(w, x, over, n, k, m, gate=over)
    assert torch.equal(over, plain * res)
