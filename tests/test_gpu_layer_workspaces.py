"""One workspace, made for the largest call, under smaller calls of the
operators around a layer's projections: each gives what it gives with a
workspace of its own."""
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


def _ws(n):
    return torch.empty(n, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("most,rows", [(600, 512), (600, 1), (4200, 4095), (4200, 512), (4200, 700)])
def test_lora(most, rows):
    n, k, r = 40, 64, 20
    g = torch.Generator("cuda").manual_seed(most + rows)
    x = torch.randn((rows, k), device="cuda", generator=g)
    a = torch.randn((2, r, k), device="cuda", generator=g).half()
    b = torch.randn((2, n, r), device="cuda", generator=g).half()
    off = torch.tensor([0, rows // 2, rows], dtype=torch.int32, device="cuda")
    print("lora %d rows in a workspace for %d" % (rows, most), flush=True)
    y = []
    for ws in (_ws(q4k.q4k_lora_ws(most, r)), _ws(q4k.q4k_lora_ws(rows, r))):
        y.append(torch.full((rows, n), float("nan"), device="cuda"))
        q4k.q4k_lora(x, a, b, y[-1], off, None, n, k, r, 2, rows, ws=ws)
    assert torch.equal(*y) and bool(y[0].isfinite().all())


@pytest.mark.parametrize("most,m,topk", [(16385, 16384, 1), (2100, 2048, 8), (2100, 200, 8)])
def test_route_and_group(most, m, topk):
    E = 64
    g = torch.Generator("cuda").manual_seed(most + m)
    logits = torch.randn((m, E), device="cuda", generator=g)
    ws = _ws(q4k.q4k_moe_group_ws(most * topk, E, topk))
    ids = torch.empty((m, topk), dtype=torch.int32, device="cuda")
    w = torch.empty((m, topk), device="cuda")
    off = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    order = torch.empty(m * topk, dtype=torch.int32, device="cuda")
    print("route %d tokens in a workspace for %d" % (m, most), flush=True)
    q4k.q4k_moe_route(logits, ids, w, E, topk, m, offsets=off, order=order, ws=ws)
    want = torch.sort(ids.flatten(), stable=True)
    assert torch.equal(order, want.indices.int())
    assert torch.equal(off, torch.searchsorted(want.values, torch.arange(E + 1, device="cuda")).int())
    if topk == 1:
        off2, order2 = torch.empty_like(off), torch.empty_like(order)
        q4k.q4k_moe_group(ids, off2, order2, m, E, ws=ws)
        assert torch.equal(off, off2) and torch.equal(order, order2)
