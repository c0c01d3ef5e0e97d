"""The operators around a layer's projections on the CPU: their refusals
through the C ABI (before any HIP call, so with fake addresses), the workspace
functions, and the binding's own checks of tensors."""
import pytest

from block_quantized_decode_q4_amd import q4k

A = 0x100000
MIS = 0x100004
BIG = 2 ** 22


@pytest.fixture(scope="module")
def lib():
    return q4k.load_library()


def _norm(lib, **kw):
    a = dict(x=A, t=0, xs=0, res=A, w=A, s=A, y=A, y16=A, q=A, d=A, k=256, m=2, eps=1e-5)
    a.update(kw)
    return lib.q4k_rmsnorm(a["x"], a["t"], a["xs"], a["res"], a["w"], a["s"], a["y"], a["y16"],
                           a["q"], a["d"], a["k"], a["m"], a["eps"], None)


def test_rmsnorm_refusals(lib):
    for miss in (dict(x=None), dict(w=None), dict(q=None), dict(d=None),
                 dict(s=None, y=None, y16=None, q=None, d=None)):
        assert _norm(lib, **miss) == q4k.Q4K_ERR_NULL, miss
    for bad in (dict(m=0), dict(m=-1), dict(m=BIG), dict(k=0), dict(k=2 ** 31), dict(k=48),
                dict(xs=255), dict(xs=2 ** 41), dict(eps=-1e-5), dict(eps=float("nan")),
                dict(eps=float("inf"))):
        assert _norm(lib, **bad) == q4k.Q4K_ERR_SHAPE, bad
    assert _norm(lib, t=3) == q4k.Q4K_ERR_UNSUPPORTED
    assert _norm(lib, t=-1) == q4k.Q4K_ERR_UNSUPPORTED
    for p in ("x", "res", "w", "s", "y", "y16", "q", "d"):
        assert _norm(lib, **{p: MIS}) == q4k.Q4K_ERR_ALIGN, p


def _route(lib, **kw):
    a = dict(l=A, ls=0, ids=A, w=A, off=A, ord=A, e=64, topk=8, m=2, ws=None, wsb=0)
    a.update(kw)
    return lib.q4k_moe_route(a["l"], a["ls"], a["ids"], a["w"], a["off"], a["ord"], a["e"],
                             a["topk"], 1, a["m"], a["ws"], a["wsb"], None)


def test_route_refusals(lib):
    for miss in (dict(l=None), dict(ids=None), dict(w=None), dict(off=None), dict(ord=None)):
        assert _route(lib, **miss) == q4k.Q4K_ERR_NULL, miss
    for bad in (dict(m=0), dict(m=BIG), dict(m=BIG // 8), dict(e=0), dict(e=1025), dict(topk=0),
                dict(topk=33), dict(topk=65, e=64), dict(topk=5, e=4), dict(ls=63),
                dict(ls=2 ** 41)):
        assert _route(lib, **bad) == q4k.Q4K_ERR_SHAPE, bad
    for p in ("l", "ids", "w", "off", "ord", "ws"):
        assert _route(lib, **{p: MIS}) == q4k.Q4K_ERR_ALIGN, p
    need = q4k.q4k_moe_group_ws(4096 * 8, 64, 8)
    assert need > 0
    assert _route(lib, m=4096) == q4k.Q4K_ERR_NULL                       # no workspace
    assert _route(lib, m=4096, ws=A, wsb=need - 1) == q4k.Q4K_ERR_SIZE


def test_group_refusals(lib):
    g = lib.q4k_moe_group
    for args in ((None, A, A), (A, None, A), (A, A, None)):
        assert g(*args, 10, 4, None, 0, None) == q4k.Q4K_ERR_NULL
    for count, groups in ((0, 4), (-1, 4), (BIG, 4), (10, 0), (10, 1025)):
        assert g(A, A, A, count, groups, None, 0, None) == q4k.Q4K_ERR_SHAPE, (count, groups)
    for args in ((MIS, A, A), (A, MIS, A), (A, A, MIS)):
        assert g(*args, 10, 4, None, 0, None) == q4k.Q4K_ERR_ALIGN
    need = q4k.q4k_moe_group_ws(10000, 4, 1)
    assert g(A, A, A, 10000, 4, None, 0, None) == q4k.Q4K_ERR_NULL
    assert g(A, A, A, 10000, 4, A, need - 1, None) == q4k.Q4K_ERR_SIZE


def test_combine_refusals(lib):
    c = lib.q4k_moe_combine
    assert c(None, A, A, A, A, 64, 2, 3, None) == q4k.Q4K_ERR_NULL
    assert c(A, None, A, A, A, 64, 2, 3, None) == q4k.Q4K_ERR_NULL
    assert c(A, A, A, A, None, 64, 2, 3, None) == q4k.Q4K_ERR_NULL
    for n, topk, m in ((0, 2, 3), (64, 0, 3), (64, 33, 3), (64, 2, 0), (64, 2, BIG),
                       (2 ** 30, 2, 1024), (2 ** 31, 2, 1)):
        assert c(A, A, A, A, A, n, topk, m, None) == q4k.Q4K_ERR_SHAPE, (n, topk, m)
    for i in range(5):
        args = [A] * 5
        args[i] = MIS
        assert c(*args, 64, 2, 3, None) == q4k.Q4K_ERR_ALIGN, i


def _grouped(lib, name, **kw):
    a = dict(w=A, x=A, d=A, y=A, off=A, xr=A, yr=A, n=100, k=512, groups=4, rows=9, div=2, xc=5,
             yc=9, ws=A, wsb=q4k.q4k_gemv_grouped_ws(512, 9))
    a.update(kw)
    rows = (a["off"], a["xr"], a["yr"], a["n"], a["k"], a["groups"], a["rows"], a["div"], a["xc"],
            a["yc"])
    if name == "f32":
        return lib.q4k_gemv_grouped(a["w"], a["x"], a["y"], *rows, a["ws"], a["wsb"], None)
    if name == "q8":
        return lib.q4k_gemv_grouped_q8(a["w"], a["x"], a["d"], a["y"], *rows, a["ws"], a["wsb"],
                                       None)
    return lib.q4k_f16_gemm_grouped(a["w"], a["x"], a["y"], *rows, None)


@pytest.mark.parametrize("name", ["f32", "q8", "f16"])
def test_grouped_refusals(lib, name):
    for p in ("w", "x", "y", "off") + (("d",) if name == "q8" else ()) + \
            (("ws",) if name != "f16" else ()):
        assert _grouped(lib, name, **{p: None}) == q4k.Q4K_ERR_NULL, p
        assert _grouped(lib, name, **{p: MIS}) == q4k.Q4K_ERR_ALIGN, p
    for p in ("xr", "yr"):
        assert _grouped(lib, name, **{p: MIS}) == q4k.Q4K_ERR_ALIGN, p
    for bad in (dict(n=0), dict(n=2 ** 31), dict(k=0), dict(groups=0), dict(groups=BIG),
                dict(rows=0), dict(rows=BIG), dict(div=0), dict(xc=0), dict(xc=BIG), dict(yc=0),
                dict(yc=BIG), dict(n=2 ** 30, rows=2 ** 21)):
        assert _grouped(lib, name, **bad) == q4k.Q4K_ERR_SHAPE, bad
    if name == "f16":
        assert _grouped(lib, name, k=96) == q4k.Q4K_ERR_UNSUPPORTED
    else:
        assert _grouped(lib, name, k=384) == q4k.Q4K_ERR_SHAPE
        assert _grouped(lib, name, k=2 ** 24 + 256, wsb=2 ** 62) == q4k.Q4K_ERR_SHAPE
        assert _grouped(lib, name, wsb=q4k.q4k_gemv_grouped_ws(512, 9) - 1) == q4k.Q4K_ERR_SIZE


def _lora(lib, **kw):
    a = dict(x=A, t=0, a=A, b=A, base=A, y=A, ranks=A, sc=A, off=A, ord=A, n=100, k=64, r=8,
             ad=3, rows=5, ws=A, wsb=q4k.q4k_lora_ws(5, 8))
    a.update(kw)
    return lib.q4k_lora(a["x"], a["t"], a["a"], a["b"], a["base"], a["y"], a["ranks"], a["sc"],
                        a["off"], a["ord"], a["n"], a["k"], a["r"], a["ad"], a["rows"], a["ws"],
                        a["wsb"], None)


def test_lora_refusals(lib):
    for p in ("x", "a", "b", "y", "off", "ws"):
        assert _lora(lib, **{p: None}) == q4k.Q4K_ERR_NULL, p
    for p in ("x", "a", "b", "base", "y", "ranks", "sc", "off", "ord", "ws"):
        assert _lora(lib, **{p: MIS}) == q4k.Q4K_ERR_ALIGN, p
    for bad in (dict(n=0), dict(n=BIG), dict(k=0), dict(k=2 ** 31), dict(r=0), dict(r=1025),
                dict(ad=0), dict(ad=BIG), dict(rows=0), dict(rows=BIG),
                dict(n=2 ** 20, rows=2 ** 21)):
        assert _lora(lib, **bad) == q4k.Q4K_ERR_SHAPE, bad
    assert _lora(lib, t=3) == q4k.Q4K_ERR_UNSUPPORTED
    assert _lora(lib, k=60) == q4k.Q4K_ERR_UNSUPPORTED
    assert _lora(lib, wsb=q4k.q4k_lora_ws(5, 8) - 1) == q4k.Q4K_ERR_SIZE


def test_workspace_bytes():
    assert q4k.q4k_moe_group_ws(1, 1, 1) == 0                  # few slots need none
    for slots, groups, topk in ((0, 4, 1), (10, 0, 1), (10, 1025, 1), (10, 4, 5), (BIG, 4, 1)):
        assert q4k.q4k_moe_group_ws(slots, groups, topk) == 0
    # counts per chunk and group; about 256 chunks at most
    assert 0 < q4k.q4k_moe_group_ws(BIG - 1, 1024, 1) <= 257 * 1024 * 4
    # x as two halves, its sub-blocks' sums as two halves, an exponent per position
    assert q4k.q4k_gemv_grouped_ws(512, 3) == 3 * (512 * 4 + 16 * 4 + 4)
    assert q4k.q4k_gemv_grouped_ws(500, 3) == 0 and q4k.q4k_gemv_grouped_ws(512, 0) == 0
    # A x in f32, the ranks in whole tiles of 16, by parts of k for few rows
    assert q4k.q4k_lora_ws(5, 17) == 4 * 5 * 32 * 4
    assert q4k.q4k_lora_ws(10000, 17) == 10000 * 32 * 4
    assert q4k.q4k_lora_ws(0, 8) == 0 and q4k.q4k_lora_ws(5, 1025) == 0


def test_binding_refuses_tensors_off_the_gpu():
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 256)
    with pytest.raises(ValueError):
        q4k.q4k_rmsnorm(x, torch.ones(256), 256, 2, y=torch.empty(2, 256))
    with pytest.raises(ValueError):
        q4k.q4k_moe_combine(x, x, None, x, 256, 1, 2)
