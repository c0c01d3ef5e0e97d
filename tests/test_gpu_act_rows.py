"""Products with an epilogue where rows must not meet: grouped rows whose indices
name nothing, positions behind the last group, and NaN in one row of x.  Rows that
are computed have the bits of a call without such rows."""
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


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _grouped(kind, w, x, y, off, n, k, rows, **how):
    if kind == "q4":
        ws = torch.empty(q4k.q4k_gemv_grouped_ws(k, rows), dtype=torch.uint8, device="cuda")
        q4k.q4k_gemv_grouped_act(w, x, y, off, n, k, 3, rows, ws=ws, **how)
    else:
        q4k.q4k_f16_gemm_grouped_act(w, x, y, off, n, k, 3, rows, **how)


@pytest.mark.parametrize("kind", ["q4", "f16"])
@pytest.mark.parametrize("rows", [9, 150])
def test_indices_that_name_nothing(kind, rows):
    n, k = 200, 512
    g = torch.Generator(device="cuda").manual_seed(rows)

    def rand(*shape):
        return torch.randn(shape, device="cuda", generator=g)

    w = B.random_q4k(g, 3 * n, k) if kind == "q4" else (rand(3 * n, k) * 0.05).half()
    x = rand(rows, k) if kind == "q4" else rand(rows, k).half()
    gate, res, bias = rand(rows, n), rand(rows, n), rand(3, n)
    # the last two positions are in no group
    off = _i32([0, rows // 3, rows // 3, rows - 2])
    how = dict(act=q4k.Q4K_ACT_GELU, gate=gate, residual=res, bias=bias, x_count=rows,
               y_count=rows)
    order = torch.randperm(rows, generator=torch.Generator().manual_seed(1)).tolist()
    clean = torch.full((rows, n), 7.0, device="cuda")
    _grouped(kind, w, x, clean, off, n, k, rows, x_rows=_i32(order), y_rows=_i32(order), **how)
    xr, yr = list(order), list(order)
    xr[0], xr[3], xr[4] = -1, rows, 1 << 30
    yr[1], yr[5], yr[6] = -4, rows, (1 << 31) - 1
    y = torch.full((rows, n), 7.0, device="cuda")
    print("rows", kind, rows, flush=True)
    _grouped(kind, w, x, y, off, n, k, rows, x_rows=_i32(xr), y_rows=_i32(yr), **how)
    out = [order[p] for p in (0, 3, 4, 1, 5, 6, rows - 2, rows - 1)]
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[out] = False
    assert bool((y[out] == 7.0).all())
    assert torch.equal(y[keep], clean[keep])
    assert bool((clean[order[-2:]] == 7.0).all())


@pytest.mark.parametrize("kind", ["q4", "f16"])
@pytest.mark.parametrize("rows", [9, 150])
def test_offsets_past_the_rows(kind, rows):
    """Offsets are cut to the rows: the last group ends with them."""
    n, k = 130, 256
    g = torch.Generator(device="cuda").manual_seed(rows)
    w = B.random_q4k(g, 3 * n, k)
    x = torch.randn((rows, k), device="cuda", generator=g)
    if kind == "f16":
        w, x = (torch.randn((3 * n, k), device="cuda", generator=g) * 0.1).half(), x.half()
    ends = [torch.empty((rows, n), device="cuda") for _ in range(2)]
    for y, last in zip(ends, (rows, rows + 1000)):
        _grouped(kind, w, x, y, _i32([0, 2, 5, last]), n, k, rows, act=q4k.Q4K_ACT_SILU)
    assert torch.equal(*ends)


@pytest.mark.parametrize("m,n,k,half", [(1, 300, 1024, False), (2, 300, 2048, False),
                                        (7, 300, 1024, False), (20, 300, 1024, False),
                                        (5, 300, 512, True), (200, 300, 448, True),
                                        (700, 4096, 512, True)])
def test_nan_in_one_row_of_x(m, n, k, half):
    g = torch.Generator(device="cuda").manual_seed(m)
    x = torch.randn((m, k), device="cuda", generator=g)
    res = torch.randn((m, n), device="cuda", generator=g)
    if half:
        w, x = (torch.randn((n, k), device="cuda", generator=g) * 0.1).half(), x.half()
    else:
        w = B.random_q4k(g, n, k)

    def call(x):
        y = torch.empty((m, n), device="cuda")
        if half:
            q4k.q4k_f16_gemm_act(w, x, y, m, n, k, act=q4k.Q4K_ACT_RELU, residual=res)
        else:
            q4k.q4k_gemv_act(w, x, y, n, k, m, act=q4k.Q4K_ACT_RELU, residual=res)
        return y

    clean = call(x)
    row = m // 2
    x[row, k // 3] = float("nan")
    y = call(x)
    assert bool(y[row].isnan().all())
    keep = torch.arange(m, device="cuda") != row
    assert torch.equal(y[keep], clean[keep])
