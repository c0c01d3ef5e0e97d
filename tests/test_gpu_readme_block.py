"""README.md's Python example of the ends of a layer's blocks, run as it stands
there, against f64 (2^-16 of the result's 2-norm, as sums in f32 allow)."""
import os
import re

import pytest

torch = pytest.importorskip("torch")

import block_ops as B  # noqa: E402
from block_quantized_decode_q4_amd import q4k  # noqa: E402

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    with open(os.path.join(ROOT, "README.md")) as f:
        code = [c for c in re.findall(r"```python\n(.*?)```", f.read(), flags=re.S)
                if "q4k_block_norm" in c]
    assert len(code) == 1
    m, k, ff, n_experts, topk = 5, 512, 768, 16, 3
    g = torch.Generator(device="cuda").manual_seed(5)

    def rand(*shape):
        return torch.randn(shape, device="cuda", generator=g)

    v = dict(q4k=q4k, m=m, k=k, ff=ff, n_experts=n_experts, topk=topk, attn=rand(m, k),
             weight=1 + 0.1 * rand(k), post=1 + 0.1 * rand(k), h=rand(m, k), y=rand(m, k),
             w_up=B.random_q4k(g, ff, k), w_gate=B.random_q4k(g, ff, k),
             w_down=B.random_q4k(g, k, ff), up=rand(m, ff), act=rand(m, ff), down_bias=rand(k),
             logits=rand(m, n_experts), balance=0.1 * rand(n_experts),
             ids=torch.empty((m, topk), dtype=torch.int32, device="cuda"),
             weights=rand(m, topk),
             offsets=torch.empty(n_experts + 1, dtype=torch.int32, device="cuda"),
             order=torch.empty(m * topk, dtype=torch.int32, device="cuda"),
             ws=torch.empty(max(16, q4k.q4k_moe_group_ws(m * topk, n_experts, topk)),
                            dtype=torch.uint8, device="cuda"))
    h = v["h"].double()
    exec(code[0], v)
    torch.cuda.synchronize()
    h = h + B.norm64(v["attn"].double(), False, v["post"], None, 1e-5)
    y = B.norm64(h, False, v["weight"], None, 1e-5)
    up = y @ B.dequantized(v["w_up"], k).double().view(ff, k).T
    gate = y @ B.dequantized(v["w_gate"], k).double().view(ff, k).T
    act = B.act64(gate, q4k.Q4K_ACT_SILU) * up
    h = h + act @ B.dequantized(v["w_down"], ff).double().view(k, ff).T + v["down_bias"].double()
    for got, want in ((v["y"], y), (v["act"], act), (v["h"], h)):
        assert float((got.double() - want).norm() / want.norm()) <= 2.0 ** -16
    ids, weights = B.route64(v["logits"].cpu().numpy(), v["balance"].cpu().numpy(), True, 4, 2,
                             topk, True, 1.0)
    assert (v["ids"].cpu().numpy() == ids).all()
    assert abs(v["weights"].cpu().numpy() - weights).max() <= 2.0 ** -23
    assert v["offsets"][-1] == m * topk
