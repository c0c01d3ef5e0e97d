"""The operators at the ends of a layer's blocks on the CPU: their refusals
through the C ABI (before any HIP call, so with fake addresses), and which
arguments the binding lets through."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from block_quantized_decode_q4_amd import q4k  # noqa: E402
from test_layer_binding_cpu import GpuTensor, _host_array, calls  # noqa: E402,F401

A = 0x100000
MIS = 0x100004
BIG = 2 ** 22


@pytest.fixture(scope="module")
def lib():
    return q4k.load_library()


def _ep(**kw):
    e = dict(bias=A, gate=A, residual=A, y=A, y16=A, gate_type=0, act=0)
    e.update(kw)
    return ctypes.addressof(_keep(q4k.q4k_epilogue(**e)))


_kept = []


def _keep(struct):
    _kept.append(struct)
    return struct


def _entries(lib):
    """Each product with an epilogue: (a call with the arguments that kw changes,
    its arguments' names of pointers that it needs)."""
    def gemv(**kw):
        a = dict(w=A, x=A, ep=_ep(), n=64, k=256, m=1)
        a.update(kw)
        return lib.q4k_gemv_act(a["w"], a["x"], a["ep"], a["n"], a["k"], a["m"], None)

    def gemm(**kw):
        a = dict(w=A, x=A, ep=_ep(), n=64, k=256, m=4)
        a.update(kw)
        return lib.q4k_f16_gemm_act(a["w"], a["x"], a["ep"], a["m"], a["n"], a["k"], None)

    def grouped(fn, with_ws):
        def call(**kw):
            a = dict(w=A, x=A, ep=_ep(), off=A, xr=A, yr=A, n=64, k=256, g=2, rows=4, div=1, xc=4,
                     yc=4, ws=A, wsb=1 << 20)
            a.update(kw)
            ws = (a["ws"], a["wsb"]) if with_ws else ()
            return fn(a["w"], a["x"], a["ep"], a["off"], a["xr"], a["yr"], a["n"], a["k"], a["g"],
                      a["rows"], a["div"], a["xc"], a["yc"], *ws, None)
        return call

    return [gemv, gemm, grouped(lib.q4k_gemv_grouped_act, True),
            grouped(lib.q4k_f16_gemm_grouped_act, False)]


@pytest.mark.parametrize("which", range(4))
def test_epilogue_refusals(lib, which):
    call = _entries(lib)[which]
    for bad in (dict(ep=None), dict(ep=_ep(y=None, y16=None)), dict(w=None), dict(x=None)):
        assert call(**bad) == q4k.Q4K_ERR_NULL, bad
    for e in (dict(act=-1), dict(act=6), dict(gate_type=q4k.Q4K_BF16), dict(gate_type=-1),
              dict(gate_type=3)):
        assert call(ep=_ep(**e)) == q4k.Q4K_ERR_UNSUPPORTED, e
    for p in ("bias", "gate", "residual", "y", "y16"):
        assert call(ep=_ep(**{p: MIS})) == q4k.Q4K_ERR_ALIGN, p
    for p in ("w", "x"):
        assert call(**{p: MIS}) == q4k.Q4K_ERR_ALIGN, p
    for bad in (dict(n=0), dict(n=2 ** 31), dict(k=0)):
        assert call(**bad) == q4k.Q4K_ERR_SHAPE, bad


def test_product_shapes(lib):
    gemv, gemm, grouped, grouped16 = _entries(lib)
    for bad in (dict(k=128), dict(k=300), dict(k=2 ** 31), dict(m=0), dict(m=-1)):
        assert gemv(**bad) == q4k.Q4K_ERR_SHAPE, bad
    assert gemv(m=33) == q4k.Q4K_ERR_UNSUPPORTED
    for bad in (dict(m=0), dict(m=2 ** 31), dict(m=2 ** 30, n=2 ** 30)):
        assert gemm(**bad) == q4k.Q4K_ERR_SHAPE, bad
    assert gemm(k=96) == q4k.Q4K_ERR_UNSUPPORTED
    for call in (grouped, grouped16):
        for bad in (dict(g=0), dict(g=BIG), dict(rows=0), dict(rows=BIG), dict(div=0),
                    dict(xc=0), dict(yc=0), dict(yc=BIG)):
            assert call(**bad) == q4k.Q4K_ERR_SHAPE, bad
        assert call(off=None) == q4k.Q4K_ERR_NULL
        for p in ("off", "xr", "yr"):
            assert call(**{p: MIS}) == q4k.Q4K_ERR_ALIGN, p
    assert grouped(ws=None) == q4k.Q4K_ERR_NULL
    assert grouped(wsb=q4k.q4k_gemv_grouped_ws(256, 4) - 1) == q4k.Q4K_ERR_SIZE
    assert grouped(k=300) == q4k.Q4K_ERR_SHAPE
    assert grouped(n=2 ** 31 - 1, rows=BIG - 1, g=BIG - 1) == q4k.Q4K_ERR_SHAPE
    assert grouped16(k=96) == q4k.Q4K_ERR_UNSUPPORTED
    assert grouped16(n=2 ** 31 - 1, rows=BIG - 1, g=BIG - 1) == q4k.Q4K_ERR_SHAPE


def _norm(lib, **kw):
    a = dict(x=A, t=0, xs=0, kind=0, pw=A, pb=A, g=A, gs=0, scale=1.0, res=A, s=A, w=A, b=A, y=A,
             y16=A, q=A, d=A, k=256, m=2, eps=1e-5)
    a.update(kw)
    return lib.q4k_block_norm(a["x"], a["t"], a["xs"], a["kind"], a["pw"], a["pb"], a["g"],
                              a["gs"], a["scale"], a["res"], a["s"], a["w"], a["b"], a["y"],
                              a["y16"], a["q"], a["d"], a["k"], a["m"], a["eps"], None)


def test_block_norm_refusals(lib):
    for miss in (dict(x=None), dict(w=None), dict(q=None), dict(d=None),
                 dict(s=None, y=None, y16=None, q=None, d=None)):
        assert _norm(lib, **miss) == q4k.Q4K_ERR_NULL, miss
    for bad in (dict(m=0), dict(m=-1), dict(m=BIG), dict(k=0), dict(k=2 ** 31), dict(k=48),
                dict(xs=255), dict(xs=2 ** 41), dict(gs=255), dict(gs=-1), dict(gs=2 ** 41),
                dict(eps=-1e-5), dict(eps=float("nan")), dict(eps=float("inf")),
                dict(scale=float("nan")), dict(scale=float("inf"))):
        assert _norm(lib, **bad) == q4k.Q4K_ERR_SHAPE, bad
    for bad in (dict(t=3), dict(t=-1), dict(kind=2), dict(kind=-1)):
        assert _norm(lib, **bad) == q4k.Q4K_ERR_UNSUPPORTED, bad
    for p in ("x", "pw", "pb", "g", "res", "s", "w", "b", "y", "y16", "q", "d"):
        assert _norm(lib, **{p: MIS}) == q4k.Q4K_ERR_ALIGN, p


def _route(lib, **kw):
    a = dict(l=A, ls=0, b=A, score=1, g=8, kg=4, ids=A, w=A, off=A, ord=A, e=64, topk=8, scale=1.0,
             m=2, ws=None, wsb=0)
    a.update(kw)
    return lib.q4k_moe_route_biased(a["l"], a["ls"], a["b"], a["score"], a["g"], a["kg"], a["ids"],
                                    a["w"], a["off"], a["ord"], a["e"], a["topk"], 1, a["scale"],
                                    a["m"], a["ws"], a["wsb"], None)


def test_route_biased_refusals(lib):
    for miss in (dict(l=None), dict(ids=None), dict(w=None), dict(off=None), dict(ord=None)):
        assert _route(lib, **miss) == q4k.Q4K_ERR_NULL, miss
    for bad in (dict(m=0), dict(m=BIG), dict(m=BIG // 8), dict(e=0), dict(e=1032), dict(topk=0),
                dict(topk=33), dict(ls=63), dict(ls=2 ** 41), dict(g=0), dict(g=65, e=65),
                dict(g=7), dict(kg=0), dict(kg=9), dict(kg=1, topk=9), dict(kg=-1),
                dict(scale=float("nan")), dict(scale=float("inf"))):
        assert _route(lib, **bad) == q4k.Q4K_ERR_SHAPE, bad
    for bad in (dict(score=2), dict(score=-1)):
        assert _route(lib, **bad) == q4k.Q4K_ERR_UNSUPPORTED, bad
    for p in ("l", "b", "ids", "w", "off", "ord", "ws"):
        assert _route(lib, **{p: MIS}) == q4k.Q4K_ERR_ALIGN, p
    need = q4k.q4k_moe_group_ws(4096 * 8, 64, 8)
    assert _route(lib, m=4096) == q4k.Q4K_ERR_NULL
    assert _route(lib, m=4096, ws=A, wsb=need - 1) == q4k.Q4K_ERR_SIZE


# ------------------------------------------------------------------ the binding
def _every_call():
    f32, f16, i32, u8, i8 = (torch.float32, torch.float16, torch.int32, torch.uint8, torch.int8)
    t = GpuTensor
    ws = t(u8, 1 << 16)
    rows = dict(y=t(f32, 5, 8), y16=t(f16, 5, 8), offsets=t(i32, 3), x_rows=t(i32, 5),
                y_rows=t(i32, 5), bias=t(f32, 2, 8), gate=t(f16, 5, 8), residual=t(f32, 5, 8))
    out = dict(y=t(f32, 3, 8), y16=t(f16, 3, 8), bias=t(f32, 8), gate=t(f32, 3, 8),
               residual=t(f32, 3, 8))
    grouped = dict(n=8, k=256, groups=2, rows=5)
    return [
        (q4k.q4k_gemv_act, dict(out, w=t(u8, 8, 144), x=t(f32, 3, 256)), dict(n=8, k=256, m=3)),
        (q4k.q4k_f16_gemm_act, dict(out, w16=t(f16, 8, 64), x16=t(f16, 3, 64)),
         dict(n=8, k=64, m=3)),
        (q4k.q4k_gemv_grouped_act, dict(rows, w=t(u8, 16, 144), x=t(f32, 5, 256), ws=ws), grouped),
        (q4k.q4k_f16_gemm_grouped_act, dict(rows, w16=t(f16, 16, 256), x16=t(f16, 5, 256)),
         grouped),
        (q4k.q4k_block_norm, dict(x=t(f32, 2, 64), weight=t(f32, 64), bias=t(f32, 64),
                                  post_weight=t(f32, 64), post_bias=t(f32, 64), gate=t(f32, 64),
                                  residual=t(f32, 2, 64), sum_out=t(f32, 2, 64), y=t(f32, 2, 64),
                                  y16=t(f16, 2, 64), q=t(i8, 2, 64), d=t(f32, 2, 2)),
         dict(k=64, m=2)),
        (q4k.q4k_moe_route_biased, dict(logits=t(f32, 2, 8), ids=t(i32, 2, 2),
                                        weights=t(f32, 2, 2), bias=t(f32, 8), offsets=t(i32, 9),
                                        order=t(i32, 4), ws=ws),
         dict(n_experts=8, topk=2, m=2)),
    ]


def test_every_entry_point_is_called(calls):                           # noqa: F811
    for call, memory, rest in _every_call():
        call(**memory, **rest)
        assert [c[0] for c in calls] == [call.__name__]
        calls.clear()


def test_arguments_that_are_refused(calls):                            # noqa: F811
    """Host arrays, tensors of another type, too short ones, ones elsewhere."""
    for call, memory, rest in _every_call():
        for name, t in memory.items():
            bad = [(_host_array(t), TypeError), (GpuTensor(torch.float64, *t.shape), TypeError)]
            if name == "ws":
                bad.pop()                      # a workspace is of any type
            else:
                bad.append((GpuTensor(t.dtype, 1), ValueError))
            away = GpuTensor(t.dtype, *t.shape)
            away.get_device = lambda: 1
            bad.append((away, ValueError))
            for value, error in bad:
                with pytest.raises(error):
                    call(**dict(memory, **{name: value}), **rest)
                assert calls == [], (call.__name__, name)


def test_one_tensor_among_addresses(calls):                            # noqa: F811
    for call, memory, rest in _every_call():
        addresses = dict.fromkeys(memory, 0x100000)
        if "ws" in memory:
            rest = dict(rest, ws_bytes=memory["ws"].numel())
        for name, t in memory.items():
            call(**dict(addresses, **{name: t}), **rest)
            assert [c[0] for c in calls] == [call.__name__], (call.__name__, name)
            calls.clear()


def test_the_gates_type(calls):                                        # noqa: F811
    """An f16 or f32 gate's type comes from its tensor, or is given beside an
    address; another than the tensor's is refused."""
    seen = []

    def take(**kw):
        q4k.q4k_gemv_act(0x100000, 0x100000, GpuTensor(torch.float32, 1, 8), 8, 256, 1, **kw)
        seen.append(calls.pop()[0])

    half, full = GpuTensor(torch.float16, 1, 8), GpuTensor(torch.float32, 1, 8)
    take(gate=half)
    take(gate=full, gate_type=q4k.Q4K_F32)
    take(gate=0x100000, gate_type=q4k.Q4K_F16)
    with pytest.raises(TypeError):
        q4k.q4k_gemv_act(0x100000, 0x100000, full, 8, 256, 1, gate=half, gate_type=q4k.Q4K_F32)
    with pytest.raises(TypeError):
        q4k.q4k_gemv_act(0x100000, 0x100000, full, 8, 256, 1, gate=GpuTensor(torch.int32, 1, 8))
    assert seen == ["q4k_gemv_act"] * 3 and calls == []
