"""Cases of the operators that finish a decoder layer's blocks: products whose
epilogue adds the bias, the activation, the gate's factor and the residual,
the norms on both sides of a residual addition, and the routing of tokens to
experts by biased scores.

Every case runs in two forms.  With ``own`` false, ``run`` computes it with
elementary torch operations in f32 (or f64); with ``own`` true it makes the
calls a user makes.  Both take the same inputs and return the same outputs.

  gemv       y = act(W x + bias) gate + residual, W in Q4_K, one to 32 vectors
  gemm       the same on an fp16 mirror of W, for prompts
  experts    the same over rows that are grouped by expert, W in Q4_K
  experts16  the same on fp16 mirrors
  norm       h = residual + scale gate N(x; after), y = N(h; before), N the
             root-mean-square or the layer norm, y in f32, in fp16 or as int8
             codes with a scale per 32 elements
  route      top-k experts by score + bias within the best groups of experts,
             their scores as weights, and the slots in the order of experts
"""
import math

import torch

own = False

_DEV = "cuda"


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one token: the attention's output projection, its bias, and the residual stream
        dict(name="projection 1 token", op="gemv", m=1, n=4096, k=4096, act="none", bias=True,
             gate=None, residual=True, out="f32"),
        # one token: the gated feed-forward block's up side
        dict(name="feed-forward 1 token", op="gemv", m=1, n=14336, k=4096, act="silu", bias=False,
             gate="f32", residual=False, out="f32"),
        # eight tokens (requests in flight, or drafted ones): the block's way down
        dict(name="feed-forward 8 tokens down", op="gemv", m=8, n=4096, k=14336, act="none",
             bias=False, gate=None, residual=True, out="f32"),
        # a prompt: the gated feed-forward block's up side, fp16 for the way down
        dict(name="feed-forward prompt", op="gemm", m=2048, n=14336, k=4096, act="silu",
             bias=False, gate="f16", residual=False, out="f16"),
        # a prompt of odd length: the way down with bias onto the residual stream
        dict(name="feed-forward prompt down", op="gemm", m=509, n=4096, k=14336, act="none",
             bias=True, gate=None, residual=True, out="f32"),
        # a decode batch on many narrow experts, gated
        dict(name="experts 16 tokens", op="experts", m=16, experts=64, topk=8, n=1536, k=2048,
             act="silu", bias=False, gate="f32", residual=False, out="f32"),
        # a prompt on eight wide experts, gated, fp16 for the way down
        dict(name="experts prompt", op="experts16", m=2048, experts=8, topk=2, n=14336, k=4096,
             act="silu", bias=False, gate="f16", residual=False, out="f16"),
        # one token between two blocks, norms on both sides, int8 for the next projection
        dict(name="norms 1 token to int8", op="norm", kind="rms", m=1, k=4096, x="f32",
             after=True, biases=False, gate="vector", scale=1.0, residual=True, out="q8"),
        # a prompt: norms on both sides, the block's output scaled, fp16 for the next projection
        dict(name="norms prompt", op="norm", kind="rms", m=4096, k=8192, x="f16", after=True,
             biases=False, gate=None, scale=0.22, residual=True, out="f16"),
        # rows of an odd width, layer norms with biases, a gate for every row
        dict(name="layer norms odd width", op="norm", kind="layer", m=1000, k=2049, x="f32",
             after=True, biases=True, gate="rows", scale=1.0, residual=True, out="f32"),
        # a decode batch: softmax scores, a bias for balance
        dict(name="route 16 tokens", op="route", m=16, experts=64, topk=6, score="softmax",
             groups=1, keep=1, renorm=False, scale=1.0),
        # a prompt: sigmoid scores, a bias, half of the groups
        dict(name="route prompt", op="route", m=8192, experts=256, topk=8, score="sigmoid",
             groups=8, keep=4, renorm=True, scale=2.5),
    ]


_ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh", "sigmoid")


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("gemv", "gemm", "experts", "experts16", "norm", "norm", "route", "route"))
    if op == "norm":
        out = rng.choice(("f32", "f16", "q8"))
        k = _log(rng, 256, 16384)
        k = max(32, k // 32 * 32) if out == "q8" else k
        m = max(1, min(_log(rng, 1, 4096), (4096 * 8192) // k))
        return dict(op=op, kind=rng.choice(("rms", "layer")), m=m, k=k,
                    x=rng.choice(("f32", "f16", "bf16")), after=rng.random() < 0.7,
                    biases=rng.random() < 0.4, gate=rng.choice((None, "vector", "rows")),
                    scale=rng.choice((1.0, 0.22)), residual=rng.random() < 0.8, out=out)
    if op == "route":
        groups = rng.choice((1, 1, 2, 4, 8))
        experts = groups * _log(rng, max(2, 8 // groups), 512 // groups)
        keep = rng.randint(1, groups)
        m = min(_log(rng, 1, 8192), 8192 * 256 // experts)
        return dict(op=op, m=m, experts=experts, topk=rng.randint(1, min(8, experts * keep // groups)),
                    score=rng.choice(("softmax", "sigmoid")), groups=groups, keep=keep,
                    renorm=rng.random() < 0.6, scale=rng.choice((1.0, 2.5)))
    how = dict(act=rng.choice(_ACTS), bias=rng.random() < 0.5,
               gate=rng.choice((None, "f32", "f16")), residual=rng.random() < 0.5,
               out=rng.choice(("f32", "f16")))
    n = _log(rng, 64, 14336)
    if op == "gemv":
        return dict(op=op, m=rng.choice((1, 1, 2, 4, rng.randint(1, 32))), n=n,
                    k=_log(rng, 1, 56) * 256, **how)
    if op == "gemm":
        return dict(op=op, m=_log(rng, 1, 2048), n=n, k=_log(rng, 1, 64) * 64, **how)
    experts = _log(rng, 4, 64)
    k = _log(rng, 1, 32) * 256
    while experts * n * k > 8 * 4096 * 14336:
        n = n // 2 + 1
    m = _log(rng, 1, 128) if op == "experts" else _log(rng, 8, 1024)
    return dict(op=op, m=m, experts=experts, topk=rng.randint(1, min(8, experts)), n=n, k=k, **how)


# ------------------------------------------------------------------ inputs
_TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=_DEV)


def _weights_q4k(g, rows, k):
    """Random Q4_K rows: any codes and 6-bit fields; d and dmin such that a
    product with a normal vector is about 2."""
    w = torch.randint(0, 256, (rows, k // 256, 144), generator=g, device=_DEV, dtype=torch.uint8)
    dd = (0.1 + torch.rand((rows, k // 256, 2), generator=g, device=_DEV)) * (0.013 / math.sqrt(k))
    w[..., 0:4] = dd.half().view(torch.uint8)
    return w.view(rows, k // 256 * 144)


def _routed(g, m, experts, topk):
    """Distinct experts per token, some experts liked more than others."""
    logits = _normal(g, m, experts) + _normal(g, experts)
    ids = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :topk]
    return ids.to(torch.int32).contiguous()


def _grouped_order(ids, groups):
    """The positions sorted by id (stable), and where each group begins."""
    flat = ids.reshape(-1).long()
    order = torch.sort(flat, stable=True).indices.to(torch.int32)
    counts = torch.bincount(flat, minlength=groups)
    offsets = torch.zeros(groups + 1, dtype=torch.int32, device=_DEV)
    offsets[1:] = counts.cumsum(0).to(torch.int32)
    return offsets, order, int(counts.max())


def prepare(case, seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(int(seed) * 6151 + 29)
    s = dict(case)
    op, m = case["op"], case["m"]
    if op == "norm":
        k = case["k"]
        s["xt"] = (_normal(g, m, k) * 2 + 0.5 * _normal(g, k)).to(_TYPES[case["x"]])
        s["res"] = _normal(g, m, k) * 4 if case["residual"] else None
        s["w_after"] = 1 + 0.1 * _normal(g, k) if case["after"] else None
        s["b_after"] = 0.1 * _normal(g, k) if case["after"] and case["biases"] else None
        s["w"] = 1 + 0.1 * _normal(g, k)
        s["b"] = 0.1 * _normal(g, k) if case["biases"] else None
        rows = {None: 0, "vector": 1, "rows": m}[case["gate"]]
        s["g"] = torch.tanh(_normal(g, rows, k)) if rows else None
        s["h"] = torch.empty((m, k), device=_DEV)
        if case["out"] == "q8":
            s["q"] = torch.empty((m, k), dtype=torch.int8, device=_DEV)
            s["d"] = torch.empty((m, k // 32), device=_DEV)
            s["values"] = torch.empty((m, k // 32, 32), dtype=torch.float16, device=_DEV)
        else:
            s["y"] = torch.empty((m, k), dtype=_TYPES[case["out"]], device=_DEV)
        return s
    if op == "route":
        experts, topk = case["experts"], case["topk"]
        s["logits"] = _normal(g, m, experts) + _normal(g, experts)
        # the bias that keeps the experts' loads alike: of the scores' size
        size = 0.1 if case["score"] == "sigmoid" else 0.5 / experts
        s["bias"] = size * _normal(g, experts)
        s["ids"] = torch.empty((m, topk), dtype=torch.int32, device=_DEV)
        s["weights"] = torch.empty((m, topk), device=_DEV)
        s["offsets"] = torch.empty(experts + 1, dtype=torch.int32, device=_DEV)
        s["order"] = torch.empty(m * topk, dtype=torch.int32, device=_DEV)
        # what grouping may need beside its outputs: far above the needed bytes
        s["ws"] = torch.empty(4 * (m * topk // 64 + 64) * (experts + 1) + 4096,
                              dtype=torch.uint8, device=_DEV)
        return s
    n, k = case["n"], case["k"]
    grouped = op in ("experts", "experts16")
    rows = m * case["topk"] if grouped else m
    mats = case["experts"] if grouped else 1
    if grouped:
        ids = _routed(g, m, mats, case["topk"])
        s["offsets"], s["order"], s["most"] = _grouped_order(ids, mats)
    x = _normal(g, m, k)
    if op in ("gemm", "experts16"):
        s["w"] = (_normal(g, mats * n, k) * (2 / math.sqrt(k))).half()
        s["x"] = x.half()
    else:
        s["w"] = _weights_q4k(g, mats * n, k)
        s["x"] = x
    s["b"] = _normal(g, mats, n) if case["bias"] else None
    s["g"] = _normal(g, rows, n).to(_TYPES[case["gate"]]) if case["gate"] else None
    s["res"] = 4 * _normal(g, rows, n) if case["residual"] else None
    s["y"] = torch.empty((rows, n), dtype=_TYPES[case["out"]], device=_DEV)
    if op == "experts":
        s["ws"] = torch.empty(rows * k * 8 + 65536, dtype=torch.uint8, device=_DEV)
    return s


# ---------------------------------------------------------------- the work
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from block_quantized_decode_q4_amd import q4k
    op, m = s["op"], s["m"]
    if op == "norm":
        out = dict(q=s["q"], d=s["d"]) if s["out"] == "q8" else \
            {"y16" if s["out"] == "f16" else "y": s["y"]}
        q4k.q4k_block_norm(
            s["xt"], s["w"], s["k"], m,
            kind=q4k.Q4K_NORM_LAYER if s["kind"] == "layer" else q4k.Q4K_NORM_RMS,
            bias=s["b"], post_weight=s["w_after"], post_bias=s["b_after"], gate=s["g"],
            gate_stride=s["k"] if s["gate"] == "rows" else 0, scale=s["scale"],
            residual=s["res"], sum_out=s["h"], eps=1e-5, **out)
        if s["out"] == "q8":
            torch.mul(s["q"].view(m, -1, 32), s["d"][..., None], out=s["values"])
            return [s["h"], s["d"], s["values"]]
        return [s["h"], s["y"]]
    if op == "route":
        q4k.q4k_moe_route_biased(
            s["logits"], s["ids"], s["weights"], s["experts"], s["topk"], m, bias=s["bias"],
            score=q4k.Q4K_SCORE_SIGMOID if s["score"] == "sigmoid" else q4k.Q4K_SCORE_SOFTMAX,
            groups=s["groups"], topk_groups=s["keep"], renorm=s["renorm"], scale=s["scale"],
            offsets=s["offsets"], order=s["order"], ws=s["ws"])
        return [s["ids"], s["weights"], s["offsets"], s["order"]]
    n, k = s["n"], s["k"]
    act = {"none": q4k.Q4K_ACT_NONE, "relu": q4k.Q4K_ACT_RELU, "silu": q4k.Q4K_ACT_SILU,
           "gelu": q4k.Q4K_ACT_GELU, "gelu_tanh": q4k.Q4K_ACT_GELU_TANH,
           "sigmoid": q4k.Q4K_ACT_SIGMOID}[s["act"]]
    y, y16 = (s["y"], None) if s["out"] == "f32" else (None, s["y"])
    how = dict(act=act, bias=s["b"], gate=s["g"], residual=s["res"], y16=y16)
    if op == "gemv":
        q4k.q4k_gemv_act(s["w"], s["x"], y, n, k, m, **how)
    elif op == "gemm":
        q4k.q4k_f16_gemm_act(s["w"], s["x"], y, m, n, k, **how)
    else:
        rows = m * s["topk"]
        how.update(x_rows=s["order"], x_div=s["topk"], x_count=m)
        if op == "experts":
            q4k.q4k_gemv_grouped_act(s["w"], s["x"], y, s["offsets"], n, k, s["experts"], rows,
                                     ws=s["ws"], **how)
        else:
            q4k.q4k_f16_gemm_grouped_act(s["w"], s["x"], y, s["offsets"], n, k, s["experts"], rows,
                                         **how)
    return s["y"]


def _dequantized(w, k):
    """f32 weights of Q4_K rows (any leading shape, bytes last)."""
    b = w.view(*w.shape[:-1], k // 256, 144)
    dd = b[..., 0:4].contiguous().view(torch.float16).float()
    lo, mid, hi = b[..., 4:8], b[..., 8:12], b[..., 12:16]
    sc = torch.cat((lo & 63, (hi & 15) | ((lo >> 6) << 4)), dim=-1).float()
    mn = torch.cat((mid & 63, (hi >> 4) | ((mid >> 6) << 4)), dim=-1).float()
    codes = b[..., 16:].reshape(*b.shape[:-1], 4, 1, 32)
    q = torch.cat((codes & 15, codes >> 4), dim=-2).reshape(*b.shape[:-1], 8, 32)
    out = (dd[..., 0:1] * sc)[..., None] * q - (dd[..., 1:2] * mn)[..., None]
    return out.view(*w.shape[:-1], k)


def _activated(z, act):
    if act == "relu":
        return torch.clamp(z, min=0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "sigmoid":
        return 1 / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    if act == "gelu_tanh":
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _normed(v, kind, w, b):
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    y = v * torch.rsqrt(v.square().mean(1, keepdim=True) + 1e-5) * w
    return y if b is None else y + b


def _run_plain(s):
    op, m = s["op"], s["m"]
    if op == "norm":
        # codes are decided next to their borders: those in f64
        wide = torch.float64 if s["out"] == "q8" else torch.float32
        p = s["xt"].to(wide)
        if s["after"]:
            p = _normed(p, s["kind"], s["w_after"], s["b_after"])
        if s["g"] is not None:
            p = p * s["g"]
        if s["scale"] != 1:
            p = p * s["scale"]
        h = (p if s["res"] is None else p + s["res"]).float()
        y = _normed(h.to(wide), s["kind"], s["w"], s["b"])
        if s["out"] != "q8":
            return [h, y.to(_TYPES[s["out"]])]
        y = y.float().view(m, -1, 32)
        top = y.abs().amax(2, keepdim=True)
        codes = torch.round(y * torch.where(top > 0, 127 / top, 0.0))
        return [h, (top / 127)[..., 0], (codes * (top / 127)).half()]
    if op == "route":
        # choices are decided next to their borders: in f64
        experts, topk, groups = s["experts"], s["topk"], s["groups"]
        l = s["logits"].double()
        if s["score"] == "sigmoid":
            score = 1 / (1 + torch.exp(-l))
        else:
            score = torch.exp(l - l.amax(1, keepdim=True))
            score = score / score.sum(1, keepdim=True)
        value = score + s["bias"]
        if s["keep"] < groups:
            parts = torch.sort(value.view(m, groups, -1), dim=2, descending=True).values
            best = torch.sort(parts[:, :, :2].sum(2), dim=1, descending=True, stable=True).indices
            kept = torch.zeros((m, groups), dtype=torch.bool, device=_DEV)
            kept.scatter_(1, best[:, : s["keep"]], True)
            kept = kept[:, :, None].expand(m, groups, experts // groups).reshape(m, experts)
            value = torch.where(kept, value, -math.inf)
        ids = torch.sort(value, dim=1, descending=True, stable=True).indices[:, :topk]
        weights = torch.gather(score, 1, ids)
        if s["renorm"]:
            weights = weights / weights.sum(1, keepdim=True)
        order = torch.sort(ids.reshape(-1), stable=True)
        bounds = torch.arange(experts + 1, device=_DEV)
        offsets = torch.searchsorted(order.values, bounds)
        return [ids.int(), (weights * s["scale"]).float(), offsets.int(), order.indices.int()]
    n, k = s["n"], s["k"]
    half = op in ("gemm", "experts16")
    bias = s["b"]
    if op in ("gemv", "gemm"):
        w = s["w"].float() if half else _dequantized(s["w"], k)
        z = s["x"].float() @ w.T
    else:
        rows, experts, topk = m * s["topk"], s["experts"], s["topk"]
        at = torch.arange(rows, device=_DEV)
        group = torch.searchsorted(s["offsets"], at.int(), right=True) - 1
        x = s["x"].float()[s["order"] // topk]
        w = s["w"].view(experts, n, -1)
        if rows <= experts:           # few rows: the matrices they meet, one by one
            w = w[group]
            w = w.float() if half else _dequantized(w, k)
            z = torch.bmm(w, x[:, :, None])[..., 0]
        else:                         # every matrix, its rows padded to the longest group
            w = w.float() if half else _dequantized(w, k)
            place = at - s["offsets"][group]
            padded = torch.zeros((experts, s["most"], k), device=_DEV)
            padded[group, place] = x
            z = torch.bmm(w, padded.transpose(1, 2).contiguous())[group, :, place]
        bias = None if bias is None else bias[group]
    y = _activated(z if bias is None else z + bias, s["act"])
    if s["g"] is not None:
        y = y * s["g"].float()
    if s["res"] is not None:
        y = y + s["res"]
    return y.to(_TYPES[s["out"]])


# --------------------------------------------------- what it cannot do without
def work(case):
    op, m = case["op"], case["m"]
    size = {None: 0, "f32": 4, "f16": 2, "bf16": 2, "q8": 1.125}
    if op == "norm":
        k = case["k"]
        each = size[case["x"]] + 4 + size[case["out"]] + (4 if case["residual"] else 0)
        each += 1 + 2 if case["out"] == "q8" else 0       # the product of codes and scales
        each += 4 if case["gate"] == "rows" else 0
        vectors = 1 + int(case["after"]) + int(case["gate"] == "vector")
        return {"bytes": m * k * each + 4 * k * vectors, "flops": 14 * m * k}
    if op == "route":
        return {"bytes": 4 * m * case["experts"] + 12 * m * case["topk"] + 8 * case["experts"],
                "flops": 10 * m * case["experts"]}
    n, k = case["n"], case["k"]
    rows, met = m, 1
    if op in ("experts", "experts16"):
        rows = m * case["topk"]
        met = case["experts"] * (1 - (1 - case["topk"] / case["experts"]) ** m)
    half = op in ("gemm", "experts16")
    bytes_ = met * n * (k * (2 if half else 0.5625) + (4 if case["bias"] else 0))
    bytes_ += m * k * (2 if half else 4)
    bytes_ += rows * n * (size[case["out"]] + size[case["gate"]] + (4 if case["residual"] else 0))
    return {"bytes": bytes_, "flops": 2 * rows * n * k}


# ------------------------------------------------------ the definition, in f64
def _exact_q4k(rows, k):
    """f64 weights of Q4_K rows, field by field."""
    sb = rows.reshape(-1, 144)
    d, dmin = sb[:, 0:4].contiguous().view(torch.float16).double().unbind(1)
    s = sb[:, 4:16].long()
    out = torch.empty((sb.shape[0], 256), dtype=torch.float64, device=sb.device)
    for j in range(8):
        if j < 4:
            sc, mn = s[:, j] % 64, s[:, j + 4] % 64
        else:
            sc = s[:, j + 4] % 16 + s[:, j - 4] // 64 * 16
            mn = s[:, j + 4] // 16 + s[:, j] // 64 * 16
        part = sb[:, 16 + 32 * (j // 2): 48 + 32 * (j // 2)].double()
        high = torch.floor(part / 16)
        code = part - 16 * high if j % 2 == 0 else high
        out[:, 32 * j: 32 * j + 32] = (d * sc)[:, None] * code - (dmin * mn)[:, None]
    return out.view(-1, k)


def _exact_norm(v, kind, w, b):
    k = v.shape[1]
    if kind == "layer":
        v = v - v.sum(1, keepdim=True) / k
    y = v / torch.sqrt((v * v).sum(1, keepdim=True) / k + 1e-5) * w.double()
    return y if b is None else y + b.double()


def _exact_act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.where(z > 0, z, 0.0)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    s = torch.sigmoid(z)
    return s if act == "sigmoid" else z * s


def exact(case, seed):
    s = prepare(case, seed)
    op, m = case["op"], case["m"]
    if op == "norm":
        k = case["k"]
        h = s["xt"].double()
        if case["after"]:
            h = _exact_norm(h, case["kind"], s["w_after"], s["b_after"])
        h = h * case["scale"]
        if s["g"] is not None:
            h = h * s["g"].double()
        if s["res"] is not None:
            h = h + s["res"].double()
        y = _exact_norm(h, case["kind"], s["w"], s["b"])
        if case["out"] != "q8":
            return [h, y]
        y = y.view(m, -1, 32)
        d = y.abs().max(2).values / 127
        return [h, d, torch.round(y / d[..., None]) * d[..., None]]
    if op == "route":
        groups, each = case["groups"], case["experts"] // case["groups"]
        l = s["logits"].double()
        score = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, dim=1)
        value = (score + s["bias"].double()).view(m, groups, each)
        first = value.max(2)
        second = value.scatter(2, first.indices[..., None], -math.inf).max(2).values
        held = first.values + (second if each > 1 else 0)
        left = torch.ones((m, groups), dtype=torch.bool, device=_DEV)
        for _ in range(groups - case["keep"]):       # the lowest group goes, the last of equal ones
            low = torch.where(left, held, math.inf).flip(1).min(1).indices
            left[torch.arange(m, device=_DEV), groups - 1 - low] = False
        value = torch.where(left[..., None], value, -math.inf).view(m, -1)
        chosen = []
        for _ in range(case["topk"]):
            at = value.max(1).indices
            chosen.append(score[torch.arange(m, device=_DEV), at])
            value[torch.arange(m, device=_DEV), at] = -math.inf
        w = torch.stack(chosen, dim=1)
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True)
        return [None, w * case["scale"], None, None]
    n, k = case["n"], case["k"]
    half = op in ("gemm", "experts16")
    rows = m if op in ("gemv", "gemm") else m * case["topk"]
    begin = [0, m] if op in ("gemv", "gemm") else s["offsets"].tolist()
    z = torch.empty((rows, n), dtype=torch.float64, device=_DEV)
    for e in range(len(begin) - 1):
        lo, hi = begin[e], begin[e + 1]
        if lo == hi:
            continue
        x = s["x"] if op in ("gemv", "gemm") else s["x"][s["order"][lo:hi].long() // case["topk"]]
        w = s["w"][e * n: (e + 1) * n]
        w = w.double() if half else _exact_q4k(w, k)
        z[lo:hi] = x.double() @ w.T
        if s["b"] is not None:
            z[lo:hi] += s["b"][e].double()
    y = _exact_act(z, case["act"])
    if s["g"] is not None:
        y = y * s["g"].double()
    return y if s["res"] is None else y + s["res"].double()
