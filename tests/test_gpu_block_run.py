"""The operators at the ends of a layer's blocks run together, as a decoder layer
runs them: the norms around the residual stream, the router with biased scores, the
experts' gated products and a gated block beside them, all with their epilogues, on
Q4_K weights (a decode batch) and on fp16 mirrors (a prompt).  Every stage is held
to f64 from what the stage before it left; the run on another stream, captured and
replayed between eager runs, and two at once give the eager run's bits.

Stages are held to 2^-16 of their result's 2-norm (f32 sums of random terms are off
by a few 2^-23 of it, activations by 2^-20; the f16 outputs by 2^-12).
"""
import numpy as np
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


class Layer:
    """One layer's weights, buffers and run."""

    def __init__(self, m, k, ff, experts, topk, parts, keep, half, seed):
        self.m, self.k, self.ff, self.experts, self.topk = m, k, ff, experts, topk
        self.parts, self.keep, self.half = parts, keep, half
        g = torch.Generator(device="cuda").manual_seed(seed)

        def rand(*shape):
            return torch.randn(shape, device="cuda", generator=g)

        def rows(n, kk):
            if half:
                return (rand(n, kk) * (2 / kk ** 0.5)).half()
            return B.random_q4k(g, n, kk)

        self.w = dict(router=rows(experts, k), up=rows(experts * ff, k),
                      gate=rows(experts * ff, k), down=rows(experts * k, ff), s_up=rows(ff, k),
                      s_gate=rows(ff, k), s_down=rows(k, ff))
        self.v = dict(post=1 + 0.1 * rand(k), norm=1 + 0.1 * rand(k), bias=0.1 * rand(experts),
                      up_bias=0.1 * rand(experts, ff), down_bias=0.1 * rand(k))
        self.x, self.stream0 = rand(m, k).half(), 2 * rand(m, k)
        slots = m * topk

        def f32(*shape):
            return torch.empty(shape, device="cuda")

        def i32(*shape):
            return torch.empty(shape, dtype=torch.int32, device="cuda")

        def act(*shape):
            return torch.empty(shape, device="cuda", dtype=torch.float16 if half else torch.float32)

        self.o = dict(h=f32(m, k), y=act(m, k), logits=f32(m, experts), ids=i32(m, topk),
                      weights=f32(m, topk), offsets=i32(experts + 1), order=i32(slots),
                      up=act(slots, ff), act=act(slots, ff), down=f32(slots, k), out=f32(m, k),
                      s_up=act(m, ff), s_act=act(m, ff), s_out=f32(m, k))

        def ws(n):
            return torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")

        self.ws_group = ws(q4k.q4k_moe_group_ws(slots, experts, topk))
        self.ws_up = ws(q4k.q4k_gemv_grouped_ws(k, slots)) if not half else None
        self.ws_down = ws(q4k.q4k_gemv_grouped_ws(ff, slots)) if not half else None

    def product(self, w, x, out, n, k, **how):
        y, y16 = (None, out) if out.dtype is torch.float16 else (out, None)
        if self.half:
            q4k.q4k_f16_gemm_act(self.w[w], x, y, self.m, n, k, y16=y16, **how)
        else:
            q4k.q4k_gemv_act(self.w[w], x, y, n, k, self.m, y16=y16, **how)

    def grouped(self, w, x, out, n, k, ws, **how):
        y, y16 = (None, out) if out.dtype is torch.float16 else (out, None)
        slots = self.m * self.topk
        if self.half:
            q4k.q4k_f16_gemm_grouped_act(self.w[w], x, y, self.o["offsets"], n, k, self.experts,
                                         slots, y16=y16, **how)
        else:
            q4k.q4k_gemv_grouped_act(self.w[w], x, y, self.o["offsets"], n, k, self.experts, slots,
                                     y16=y16, ws=ws, **how)

    def run(self):
        o, v, m, k, ff = self.o, self.v, self.m, self.k, self.ff
        q4k.q4k_block_norm(self.x, v["norm"], k, m, post_weight=v["post"], scale=0.5,
                           residual=self.stream0, sum_out=o["h"],
                           **{"y16" if self.half else "y": o["y"]})
        self.product("router", o["y"], o["logits"], self.experts, k)
        q4k.q4k_moe_route_biased(o["logits"], o["ids"], o["weights"], self.experts, self.topk, m,
                                 bias=v["bias"], score=q4k.Q4K_SCORE_SIGMOID, groups=self.parts,
                                 topk_groups=self.keep, scale=1.5, offsets=o["offsets"],
                                 order=o["order"], ws=self.ws_group)
        by_token = dict(x_rows=o["order"], x_div=self.topk, x_count=m)
        self.grouped("up", o["y"], o["up"], ff, k, self.ws_up, bias=v["up_bias"], **by_token)
        self.grouped("gate", o["y"], o["act"], ff, k, self.ws_up, act=q4k.Q4K_ACT_SILU,
                     gate=o["up"], **by_token)
        self.grouped("down", o["act"], o["down"], k, ff, self.ws_down, y_rows=o["order"])
        q4k.q4k_moe_combine(o["down"], o["weights"], o["ids"], o["out"], k, self.topk, m,
                            residual=o["h"])
        # the block that all tokens take: onto the experts' sum, in place
        self.product("s_up", o["y"], o["s_up"], ff, k)
        self.product("s_gate", o["y"], o["s_act"], ff, k, act=q4k.Q4K_ACT_GELU_TANH, gate=o["s_up"])
        o["s_out"].copy_(o["out"])
        self.product("s_down", o["s_act"], o["s_out"], k, ff, bias=v["down_bias"],
                     residual=o["s_out"])

    def outputs(self):
        torch.cuda.synchronize()
        return {n: t.cpu().numpy().copy() for n, t in self.o.items()}

    def weights64(self, name, n, k):
        w = self.w[name]
        return (w.double() if self.half else B.dequantized(w, k)).view(-1, n, k)


#         m, k, ff, experts, topk, groups, kept, fp16 mirrors, seed
LAYERS = [(1, 512, 768, 8, 2, 4, 2, False, 1), (5, 512, 768, 6, 2, 1, 1, False, 2),
          (30, 256, 512, 40, 4, 8, 3, False, 3), (70, 512, 768, 8, 2, 4, 2, True, 4),
          (300, 256, 320, 16, 3, 2, 1, True, 5)]


def _close(got, want, what, size):
    got = got.double()
    off = float((got - want).norm() / want.norm())
    assert off <= size, (what, off)


@pytest.mark.parametrize("shape", LAYERS)
def test_stages(shape):
    layer = Layer(*shape)
    print("layer", shape, flush=True)
    layer.run()
    o, v, m, k, ff, topk = layer.o, layer.v, layer.m, layer.k, layer.ff, layer.topk
    f32 = 2.0 ** -16
    act = 2.0 ** -11 if layer.half else f32
    p = B.norm64(layer.x.double(), False, v["post"], None, 1e-5)
    h = layer.stream0.double() + 0.5 * p
    _close(o["h"], h, "h", f32)
    _close(o["y"], B.norm64(o["h"].double(), False, v["norm"], None, 1e-5), "y", act)
    y = o["y"].double()
    _close(o["logits"], y @ layer.weights64("router", layer.experts, k)[0].T, "logits", f32)
    ids, weights = B.route64(o["logits"].cpu().numpy(), v["bias"].cpu().numpy(), True, layer.parts,
                             layer.keep, topk, True, 1.5)
    assert np.array_equal(o["ids"].cpu().numpy(), ids)
    assert np.allclose(o["weights"].cpu().numpy(), weights, rtol=2.0 ** -23, atol=0)
    flat = ids.reshape(-1)
    pos = np.argsort(flat, kind="stable")
    assert np.array_equal(o["order"].cpu().numpy(), pos)
    pos_t = torch.from_numpy(pos).cuda()
    expert = torch.from_numpy(flat[pos]).long().cuda()
    x = y[pos_t // topk]
    up = torch.stack([layer.weights64("up", ff, k)[e] @ r for e, r in zip(expert, x)])
    _close(o["up"], up + v["up_bias"].double()[expert], "up", act)
    gate = torch.stack([layer.weights64("gate", ff, k)[e] @ r for e, r in zip(expert, x)])
    _close(o["act"], B.act64(gate, q4k.Q4K_ACT_SILU) * o["up"].double(), "act", act)
    down = torch.empty((m * topk, k), device="cuda", dtype=torch.float64)
    down[pos_t] = torch.stack([layer.weights64("down", k, ff)[e] @ r
                               for e, r in zip(expert, o["act"].double())])
    _close(o["down"], down, "down", f32)
    out = (o["down"].double().view(m, topk, k) * o["weights"].double()[..., None]).sum(1)
    _close(o["out"], out + o["h"].double(), "out", f32)
    _close(o["s_up"], y @ layer.weights64("s_up", ff, k)[0].T, "s_up", act)
    z = y @ layer.weights64("s_gate", ff, k)[0].T
    _close(o["s_act"], B.act64(z, q4k.Q4K_ACT_GELU_TANH) * o["s_up"].double(), "s_act", act)
    z = o["s_act"].double() @ layer.weights64("s_down", k, ff)[0].T + v["down_bias"].double()
    _close(o["s_out"], z + o["out"].double(), "s_out", f32)


@pytest.mark.parametrize("shape", LAYERS)
def test_stream_and_graph(shape):
    layer = Layer(*shape)
    layer.run()
    eager = layer.outputs()

    def same(what):
        now = layer.outputs()
        for n in eager:
            assert np.array_equal(now[n].view(np.uint8), eager[n].view(np.uint8)), (what, n)
            layer.o[n].view(torch.uint8).fill_(0x7F)

    same("eager")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.run()
    torch.cuda.current_stream().wait_stream(side)
    same("another stream")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        layer.run()
    for i in range(3):
        graph.replay()
        same("replay %d" % i)
        layer.run()
        same("eager after replay %d" % i)
    graph.replay()
    graph.replay()
    same("two replays in a row")


def test_two_at_once():
    layers = [Layer(7, 512, 768, 6, 2, 3, 2, False, 11), Layer(90, 512, 1024, 8, 3, 4, 4, True, 12)]
    alone = []
    for layer in layers:
        layer.run()
        alone.append(layer.outputs())
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    for _ in range(5):
        for layer, stream in zip(layers, streams):
            with torch.cuda.stream(stream):
                layer.run()
    for layer, ref in zip(layers, alone):
        now = layer.outputs()
        for n in ref:
            assert np.array_equal(now[n].view(np.uint8), ref[n].view(np.uint8)), n


def test_explicit_stream_argument():
    n, k = 300, 512
    g = torch.Generator(device="cuda").manual_seed(1)
    w, x = B.random_q4k(g, n, k), torch.randn((3, k), device="cuda", generator=g)
    ref, y = torch.empty((3, n), device="cuda"), torch.empty((3, n), device="cuda")
    q4k.q4k_gemv_act(w, x, ref, n, k, 3, act=q4k.Q4K_ACT_SILU)
    s = torch.cuda.Stream()
    for how in (s, s.cuda_stream):
        y.zero_()
        torch.cuda.synchronize()
        q4k.q4k_gemv_act(w, x, y, n, k, 3, act=q4k.Q4K_ACT_SILU, stream=how)
        s.synchronize()
        assert torch.equal(y, ref)
