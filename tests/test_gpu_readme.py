"""The README's example around a layer's projections, run as it stands there and
held to f64: up is act here (no activation between), and the weights of the
fp16 products are those of the Q4_K ones."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from block_quantized_decode_q4_amd import q4k, synth  # noqa: E402
from readme_calls import blocks  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m", [1, 9])
def test_layer_example(oracle_mod, m):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lib = q4k.load_library()
    k, ff, E, topk, n, r, adapters = 512, 768, 6, 2, 96, 8, 3
    slots = m * topk
    rng = np.random.default_rng(m)

    def f32(*shape):
        return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).cuda()

    def i32(*shape):
        return torch.full(shape, -7, dtype=torch.int32, device="cuda")

    w_up, w_down = (torch.from_numpy(synth.make_inputs(E * rows, kk, 1, seed, (1e-5, 1e-3))[0]).cuda()
                    for rows, kk, seed in ((ff, k, 1), (k, ff, 2)))
    t = dict(x=f32(m, k).half(), res=f32(m, k), w=f32(k), y=f32(m, k), y16=f32(m, k).half(),
             q=torch.zeros((m, k), dtype=torch.int8, device="cuda"), d=f32(m, k // 32),
             logits=f32(m, E), ids=i32(m, topk), wts=f32(m, topk), offsets=i32(E + 1),
             order=i32(slots), W_up=w_up, W_down=w_down, up=f32(slots, ff), down=f32(slots, k),
             W16_up=torch.empty((E * ff, k), dtype=torch.float16, device="cuda"), out=f32(m, k),
             adapter_ids=torch.from_numpy(rng.integers(-1, adapters, m).astype(np.int32)).cuda(),
             a_offsets=i32(adapters + 1), a_order=i32(m), A=f32(adapters, r, k).half(),
             B=f32(adapters, n, r).half(), proj=f32(m, n), scales=f32(adapters),
             ranks=torch.tensor([8, 3, 5], dtype=torch.int32, device="cuda"))
    t["act"] = t["up"]
    ws_bytes = max(q4k.q4k_moe_group_ws(slots, E, topk), q4k.q4k_moe_group_ws(m, adapters),
                   q4k.q4k_gemv_grouped_ws(max(k, ff), slots), q4k.q4k_lora_ws(m, r))
    t["ws"] = torch.empty(ws_bytes, dtype=torch.uint8, device="cuda")
    q4k.q4k_mirror_f16(w_up, t["W16_up"], E * ff, k)
    start = {name: t[name].cpu().numpy().astype(np.float64) for name in ("x", "res", "proj")}
    env = {name: ctypes.c_void_p(v.data_ptr()) for name, v in t.items()}
    env.update(k=k, m=m, E=E, ff=ff, topk=topk, slots=slots, n=n, r=r, adapters=adapters, eps=1e-5,
               ws_bytes=ws_bytes, stream=torch.cuda.current_stream().cuda_stream, NULL=None,
               Q4K_F16=q4k.Q4K_F16)
    for name, args in blocks()[1]:
        print("readme m=%d %s" % (m, name), flush=True)
        values = [env[a] if a in env else int(a) for a in args.values()]
        assert getattr(lib, name)(*values) == q4k.Q4K_OK
    torch.cuda.synchronize()
    o = {name: v.cpu().numpy() for name, v in t.items()}

    h = (start["x"].astype(np.float32) + start["res"].astype(np.float32))
    assert np.array_equal(o["res"], h)
    y16 = o["y16"].astype(np.float64)
    h = h.astype(np.float64)
    y = h / np.sqrt((h * h).mean(1, keepdims=True) + 1e-5) * o["w"]
    # y within two roundings of f32, y16 one more of fp16 (or of its subnormals)
    assert (np.abs(y16 - y) <= (2.0 ** -11 + 2.0 ** -22) * np.abs(y) + 2.0 ** -25).all()
    up = o["W16_up"].astype(np.float64).reshape(E, ff, k)
    down = oracle_mod.dequant(o["W_down"], E * k, ff).astype(np.float64).reshape(E, k, ff)
    out = h.copy()
    ids = np.argsort(-o["logits"], axis=1, kind="stable")[:, :topk]
    p = np.exp(np.take_along_axis(o["logits"].astype(np.float64), ids, 1))
    p /= p.sum(1, keepdims=True)
    for i in range(m):
        for j in range(topk):
            out[i] += p[i, j] * (down[ids[i, j]] @ (up[ids[i, j]] @ y16[i]))
    # random data, so the f32 roundings (at most 2^-23 of a term, a few hundred per
    # sum and two sums in a row) add like a random walk: 2^-18 of the result's norm
    assert np.linalg.norm(o["out"] - out) <= 2.0 ** -18 * np.linalg.norm(out)
    for i, a in enumerate(o["adapter_ids"]):
        want, mag = start["proj"][i], np.abs(start["proj"][i])
        tol = 0
        if a >= 0:
            A, B = (o[s][a].astype(np.float64) for s in "AB")
            A, B, s = A[: o["ranks"][a]], B[:, : o["ranks"][a]], float(o["scales"][a])
            v = A @ y16[i]
            want = want + s * (B @ v)
            mag = mag + abs(s) * (np.abs(B) @ (np.abs(A) @ np.abs(y16[i])))
            tol = 2.0 ** -38 * abs(s) * np.abs(B).sum(1) * np.abs(v).max()
        assert (np.abs(o["proj"][i] - want) <= (k + r + 4) * 2.0 ** -23 * mag + tol).all(), i
