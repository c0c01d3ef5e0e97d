"""The operators around the projections run together, as a decoder layer runs
them: norm with residual and Q8 output, a shared Q4_K projection with adapters
beside it, the router, the experts' up and down products and their weighted
sum.  Every stage is held to its own tolerance against f64 from what the stage
before it left on the GPU; the whole run on another stream, and captured into
a graph and replayed between eager runs, gives the eager run's bits.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from block_quantized_decode_q4_amd import q4k, synth  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    q4k.load_library()
    yield


class Layer:
    """One layer's weights, buffers and run."""

    def __init__(self, m, k, ff, experts, topk, r, adapters, seed):
        self.m, self.k, self.ff, self.experts, self.topk = m, k, ff, experts, topk
        self.r, self.adapters = r, adapters
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)

        def rows(n, kk):
            return torch.from_numpy(synth.make_inputs(n, kk, 1, int(rng.integers(1 << 30)),
                                                      (1e-5, 1e-3))[0]).cuda()

        def rand(*shape):
            return torch.randn(shape, device="cuda", generator=g)

        self.w = dict(proj=rows(k, k), router=rows(experts, k), up=rows(experts * ff, k),
                      gate=rows(experts * ff, k), down=rows(experts * k, ff))
        self.norm = 1 + 0.1 * rand(k)
        self.a = (rand(adapters, r, k) * 0.05).half()
        self.b = (rand(adapters, k, r) * 0.05).half()
        self.scales = torch.full((adapters,), 0.5, device="cuda")
        self.ids = torch.from_numpy(rng.integers(-1, adapters, size=m).astype(np.int32)).cuda()
        self.x = rand(m, k).half()
        self.stream0 = rand(m, k)
        slots = m * topk

        def f32(*shape):
            return torch.empty(shape, device="cuda")

        def i32(*shape):
            return torch.empty(shape, dtype=torch.int32, device="cuda")

        def ws(n):
            return torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")

        self.o = dict(h=f32(m, k), y=f32(m, k), q=torch.empty((m, k), dtype=torch.int8, device="cuda"),
                      d=f32(m, k // 32), proj=f32(m, k), logits=f32(m, experts), eids=i32(m, topk),
                      ew=f32(m, topk), eoff=i32(experts + 1), eorder=i32(slots),
                      aoff=i32(adapters + 1), aorder=i32(m), up=f32(slots, ff), gate=f32(slots, ff),
                      act=f32(slots, ff), down=f32(slots, k), out=f32(m, k))
        self.ws_group = ws(max(q4k.q4k_moe_group_ws(slots, experts, topk),
                               q4k.q4k_moe_group_ws(m, adapters, 1)))
        self.ws_lora = ws(q4k.q4k_lora_ws(m, r))
        self.ws_up = ws(q4k.q4k_gemv_grouped_ws(k, slots))
        self.ws_down = ws(q4k.q4k_gemv_grouped_ws(ff, slots))

    def run(self):
        o, w, m, k, ff = self.o, self.w, self.m, self.k, self.ff
        slots = m * self.topk
        q4k.q4k_rmsnorm(self.x, self.norm, k, m, residual=self.stream0, sum_out=o["h"], y=o["y"],
                        q=o["q"], d=o["d"])
        q4k.q4k_gemv(w["proj"], o["y"], o["proj"], k, k, m)
        q4k.q4k_moe_group(self.ids, o["aoff"], o["aorder"], m, self.adapters, ws=self.ws_group)
        q4k.q4k_lora(o["y"], self.a, self.b, o["proj"], o["aoff"], o["aorder"], k, k, self.r,
                     self.adapters, m, base=o["proj"], scales=self.scales, ws=self.ws_lora)
        q4k.q4k_gemv(w["router"], o["y"], o["logits"], self.experts, k, m)
        q4k.q4k_moe_route(o["logits"], o["eids"], o["ew"], self.experts, self.topk, m,
                          offsets=o["eoff"], order=o["eorder"], ws=self.ws_group)
        by_token = dict(x_rows=o["eorder"], x_div=self.topk, x_count=m)
        q4k.q4k_gemv_grouped(w["gate"], o["y"], o["gate"], o["eoff"], ff, k, self.experts, slots,
                             ws=self.ws_up, **by_token)
        q4k.q4k_gemv_grouped_q8(w["up"], o["q"], o["d"], o["up"], o["eoff"], ff, k, self.experts,
                                slots, ws=self.ws_up, **by_token)
        torch.sigmoid(o["gate"], out=o["act"])
        o["act"].mul_(o["gate"]).mul_(o["up"])
        q4k.q4k_gemv_grouped(w["down"], o["act"], o["down"], o["eoff"], k, ff, self.experts, slots,
                             y_rows=o["eorder"], ws=self.ws_down)
        q4k.q4k_moe_combine(o["down"], o["ew"], o["eids"], o["out"], k, self.topk, m,
                            residual=o["h"])

    def outputs(self):
        torch.cuda.synchronize()
        return {n: t.cpu().numpy().copy() for n, t in self.o.items()}


def _terms(oracle_mod, w, n, k):
    """f64 weights, and the magnitudes of their two terms bounded by the
    weight's and twice its block's min."""
    return oracle_mod.dequant(w.cpu().numpy(), n, k).astype(np.float64)


LAYERS = [(1, 512, 768, 6, 2, 4, 2, 1), (5, 512, 768, 6, 2, 8, 3, 2), (30, 256, 512, 40, 4, 16, 5, 3)]


@pytest.mark.parametrize("shape", LAYERS)
def test_layer_stages(oracle_mod, shape):
    layer = Layer(*shape)
    m, k, ff, E, topk = layer.m, layer.k, layer.ff, layer.experts, layer.topk
    print("layer", shape, flush=True)
    layer.run()
    o = layer.outputs()
    h = layer.x.float().cpu().numpy() + layer.stream0.cpu().numpy()
    assert np.array_equal(o["h"], h)
    h64 = h.astype(np.float64)
    y = h64 / np.sqrt((h64 ** 2).mean(1, keepdims=True) + 1e-5) * layer.norm.cpu().numpy()
    # eps reaches the call as f32: 2^-24 of it, far below a rounding of y
    assert (np.abs(o["y"] - y) <= 2.0 ** -22 * np.abs(y)).all()
    q_ref, d_ref = oracle_mod.quantize_q8(o["y"])
    assert np.array_equal(o["q"], q_ref) and np.array_equal(o["d"], d_ref)
    y = o["y"].astype(np.float64)
    # the shared projection (1e-5 sum |w||x|) and its adapters
    wp = _terms(oracle_mod, layer.w["proj"], k, k)
    ref, tol = y @ wp.T, 1e-5 * (np.abs(y) @ np.abs(wp).T)
    a, b = layer.a.cpu().numpy().astype(np.float64), layer.b.cpu().numpy().astype(np.float64)
    for t, i in enumerate(layer.ids.cpu().numpy()):
        if i >= 0:
            v = a[i] @ y[t]
            ref[t] += 0.5 * (b[i] @ v)
            tol[t] += (k + layer.r + 4) * 2.0 ** -23 * (
                np.abs(ref[t]) + 0.5 * (np.abs(b[i]) @ (np.abs(a[i]) @ np.abs(y[t]))))
    assert (np.abs(o["proj"] - ref) <= tol).all()
    # the router's choice from the logits it was given
    order = np.argsort(-o["logits"], axis=1, kind="stable")[:, :topk]
    assert np.array_equal(o["eids"], order)
    p = np.exp(np.take_along_axis(o["logits"], order, 1).astype(np.float64))
    assert np.allclose(o["ew"], p / p.sum(1, keepdims=True), rtol=300 * 2.0 ** -24, atol=0)
    flat = o["eids"].reshape(-1)
    pos = np.argsort(flat, kind="stable")
    assert np.array_equal(o["eorder"], pos)
    assert np.array_equal(o["eoff"], np.searchsorted(flat[pos], np.arange(E + 1)))
    # the experts, position by position (random data: 2^-18 of the row's scale)
    mats = {n: _terms(oracle_mod, layer.w[n], E * s[0], s[1]).reshape(E, *s)
            for n, s in dict(gate=(ff, k), up=(ff, k), down=(k, ff)).items()}
    xq = (o["q"].reshape(m, -1, 32).astype(np.float32) * o["d"][:, :, None]).reshape(m, k)
    act = o["act"].astype(np.float64)
    for i, slot in enumerate(pos):
        e = flat[slot]
        for got, want in ((o["gate"][i], mats["gate"][e] @ y[slot // topk]),
                          (o["up"][i], mats["up"][e] @ xq[slot // topk].astype(np.float64)),
                          (o["down"][slot], mats["down"][e] @ act[i])):
            assert np.linalg.norm(got - want) <= 2.0 ** -18 * np.linalg.norm(want)
    down = o["down"].astype(np.float64).reshape(m, topk, k) * o["ew"][:, :, None]
    mag = np.abs(down).sum(1) + np.abs(h)
    assert (np.abs(o["out"] - (down.sum(1) + h)) <= (topk + 2) * 2.0 ** -24 * mag).all()


@pytest.mark.parametrize("shape", LAYERS)
def test_layer_stream_and_graph(shape):
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


def test_two_layers_at_once():
    """Two streams, each with workspaces of its own."""
    layers = [Layer(7, 512, 768, 6, 2, 8, 3, 11), Layer(3, 512, 1024, 9, 3, 4, 2, 12)]
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
    """stream=: a torch stream or its address, also while another is current."""
    x = torch.randn((3, 256), device="cuda")
    w = torch.ones(256, device="cuda")
    ref, y = torch.empty_like(x), torch.empty_like(x)
    q4k.q4k_rmsnorm(x, w, 256, 3, y=ref)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for how in (s, s.cuda_stream):
        y.zero_()
        torch.cuda.synchronize()
        q4k.q4k_rmsnorm(x, w, 256, 3, y=y, stream=how)
        s.synchronize()
        assert torch.equal(y, ref)


def test_offsets_beyond_32_bits():
    """Rows whose byte and element offsets pass 2^31 and 2^32."""
    rng = np.random.default_rng(21)
    # Q4_K experts: the last of 4.6 GB, y rows behind 2^31 elements
    n, k, groups = 14336, 14336, 40
    row = k // 256 * 144
    w = torch.empty(groups * n * row, dtype=torch.uint8, device="cuda")
    part, x = synth.make_inputs(n, k, 2, seed=22)
    w[(groups - 1) * n * row:] = torch.from_numpy(part).cuda()
    y_count = 160000
    y = torch.empty((y_count, n), device="cuda")
    rows = torch.tensor([y_count - 1, y_count - 3], dtype=torch.int32, device="cuda")
    off = torch.zeros(groups + 1, dtype=torch.int32, device="cuda")
    off[groups] = 2
    ws = torch.empty(q4k.q4k_gemv_grouped_ws(k, 2), dtype=torch.uint8, device="cuda")
    x_d = torch.from_numpy(x).cuda()
    print("grouped, last of %d experts" % groups, flush=True)
    q4k.q4k_gemv_grouped(w, x_d, y, off, n, k, groups, 2, y_rows=rows, y_count=y_count, ws=ws)
    ref = torch.empty((2, n), device="cuda")
    q4k.q4k_gemv(w[(groups - 1) * n * row:], x_d, ref, n, k, 2)
    got = torch.stack((y[-1], y[-3]))
    assert float((got - ref).norm() / ref.norm()) <= 2.0 ** -18
    del w, y
    # fp16 experts: 5.4 GB
    n, k, groups = 16384, 16384, 10
    w = torch.empty((groups, n, k), dtype=torch.float16, device="cuda")
    w[-1] = torch.randn((n, k), device="cuda") * 0.05
    x16 = torch.randn((3, k), device="cuda").half()
    off = torch.zeros(groups + 1, dtype=torch.int32, device="cuda")
    off[groups] = 3
    y = torch.empty((3, n), device="cuda")
    print("grouped fp16, last of %d experts" % groups, flush=True)
    q4k.q4k_f16_gemm_grouped(w, x16, y, off, n, k, groups, 3)
    ref = torch.empty_like(y)
    q4k.q4k_f16_gemm(w[-1], x16, ref, 3, n, k)
    assert torch.equal(y, ref)
    del w
    # norm: 2.3 G elements, the last rows
    m, k = 70000, 32768
    x = torch.empty((m, k), dtype=torch.float16, device="cuda")
    x[-4:] = torch.randn((4, k), device="cuda").half()
    g = torch.ones(k, device="cuda")
    y16 = torch.empty((m, k), dtype=torch.float16, device="cuda")
    print("norm of %d x %d" % (m, k), flush=True)
    q4k.q4k_rmsnorm(x, g, k, m, y16=y16)
    few = torch.empty((4, k), dtype=torch.float16, device="cuda")
    q4k.q4k_rmsnorm(x[-4:].contiguous(), g, k, 4, y16=few)
    assert torch.equal(y16[-4:], few)
    del x, y16
    # adapters and combination: rows of y behind 2^32 elements
    rows, n, k, r = 1050000, 4096, 8, 8
    x = torch.zeros((rows, k), device="cuda")
    x[-1] = torch.randn(k, device="cuda")
    a = torch.randn((1, r, k), device="cuda").half()
    b = torch.randn((1, n, r), device="cuda").half()
    y = torch.empty((rows, n), device="cuda")
    off = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    order = torch.full((rows,), rows - 1, dtype=torch.int32, device="cuda")
    ws = torch.empty(q4k.q4k_lora_ws(rows, r), dtype=torch.uint8, device="cuda")
    print("adapters, row %d" % (rows - 1), flush=True)
    q4k.q4k_lora(x, a, b, y, off, order, n, k, r, 1, rows, ws=ws)
    v = a[0].double() @ x[-1].double()
    ref = b[0].double() @ v
    assert float((y[-1].double() - ref).norm() / ref.norm()) <= 2.0 ** -20
    m, topk = rows // 2, 2
    y[-2:] = torch.randn((2, n), device="cuda")
    wgt = torch.full((m, topk), 0.5, device="cuda")
    out = torch.empty((m, n), device="cuda")
    print("combination of %d rows" % (m * topk), flush=True)
    q4k.q4k_moe_combine(y, wgt, None, out, n, topk, m)
    assert torch.equal(out[-1], 0.5 * y[-2] + 0.5 * y[-1])
