"""Cases of the operators around the quantized projections of a decoder layer:
the norm in front of them, the experts' routing, products and combination, and
low-rank adapters beside them.

Every case runs in two forms.  With ``own`` false, ``run`` computes it with
elementary torch operations in f32 (or f64); with ``own`` true it makes the
calls a user makes.  Both take the same inputs and return the same outputs.

  rmsnorm    h = x + residual, y = h rsqrt(mean h^2 + eps) w, y in f32, in fp16
             or as int8 codes with a scale per 32 elements
  route      top-k experts of every token, their softmax weights, and the
             slots (token, choice) in the order of their experts
  combine    the weighted sum of each token's expert outputs
  grouped    products of rows that are grouped by expert with the expert's
             matrix: Q4_K weights with f32 or int8 activations, or an fp16
             mirror with fp16 activations
  lora       y = base + scale B (A x), a low-rank pair per request
"""
import math

import torch

own = False

_DEV = "cuda"


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one token between two layers: the residual stream is updated, and the
        # next projection takes f32 or int8 activations
        dict(name="rmsnorm 1 token to int8", op="rmsnorm", m=1, k=4096, x="f32", residual=True,
             out="q8"),
        # a prompt: the sublayer's fp16 output joins the f32 residual stream,
        # the prefill products take fp16
        dict(name="rmsnorm prompt to fp16", op="rmsnorm", m=4096, k=8192, x="f16", residual=True,
             out="f16"),
        # a small decode batch picks its experts
        dict(name="route 8 tokens", op="route", m=8, experts=64, topk=8, renorm=True),
        # a prompt picks its experts: the slots are sorted for the products
        dict(name="route prompt", op="route", m=8192, experts=128, topk=8, renorm=True),
        # the experts' outputs of a small decode batch
        dict(name="combine 4 tokens", op="combine", m=4, n=2048, topk=8, residual=True),
        # the experts' outputs of a prompt, without a residual
        dict(name="combine prompt", op="combine", m=4096, n=4096, topk=2, residual=False),
        # one token through two of eight wide experts (up projection)
        dict(name="experts 1 token f32", op="grouped", act="f32", m=1, experts=8, topk=2, n=14336,
             k=4096, side="up"),
        # a decode batch on many narrow experts, int8 activations (down projection)
        dict(name="experts batch int8", op="grouped", act="q8", m=16, experts=64, topk=8, n=2048,
             k=1536, side="down"),
        # a larger decode batch, every expert met (down projection, long rows)
        dict(name="experts batch f32", op="grouped", act="f32", m=48, experts=8, topk=2, n=4096,
             k=14336, side="down"),
        # a prompt on the fp16 mirrors of eight wide experts
        dict(name="experts prompt fp16", op="grouped", act="f16", m=2048, experts=8, topk=2,
             n=14336, k=4096, side="up"),
        # a decode batch whose requests bring their adapters, one without
        dict(name="adapters batch", op="lora", m=24, adapters=16, r=16, n=4096, k=4096, x="f32",
             ragged=True),
        # prompts of several requests in one batch, ranks up to 64
        dict(name="adapters prompt", op="lora", m=2048, adapters=8, r=64, n=4096, k=4096, x="f16",
             ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rmsnorm", "route", "combine", "grouped", "grouped", "grouped", "lora"))
    if op == "rmsnorm":
        out = rng.choice(("f32", "f16", "q8"))
        k = _log(rng, 256, 16384)
        k = max(32, k // 32 * 32) if out == "q8" else k
        m = _log(rng, 1, 4096)
        m = max(1, min(m, (4096 * 8192) // k))
        return dict(op=op, m=m, k=k, x=rng.choice(("f32", "f16", "bf16")),
                    residual=rng.random() < 0.7, out=out)
    if op == "route":
        experts = _log(rng, 4, 512)
        return dict(op=op, m=min(_log(rng, 1, 8192), 8192 * 128 // experts), experts=experts,
                    topk=rng.randint(1, min(8, experts)), renorm=rng.random() < 0.5)
    if op == "combine":
        n, topk = _log(rng, 256, 8192), rng.randint(1, 8)
        m = max(1, min(_log(rng, 1, 4096), 4096 * 4096 * 2 // (n * topk)))
        return dict(op=op, m=m, n=n, topk=topk, residual=rng.random() < 0.5)
    if op == "lora":
        return dict(op=op, m=_log(rng, 1, 2048), adapters=_log(rng, 1, 32), r=rng.randint(4, 64),
                    n=_log(rng, 256, 4096), k=_log(rng, 8, 128) * 32, x=rng.choice(("f32", "f16")),
                    ragged=rng.random() < 0.5)
    act = rng.choice(("f32", "q8", "f16"))
    experts = _log(rng, 4, 64)
    n = _log(rng, 128, 8192)
    k = _log(rng, 1, 32) * 256
    while experts * n * k > 8 * 4096 * 14336:
        n = n // 2 + 1
    return dict(op=op, act=act, m=_log(rng, 8, 1024) if act == "f16" else _log(rng, 1, 128),
                experts=experts, topk=rng.randint(1, min(8, experts)), n=n, k=k,
                side=rng.choice(("up", "down")))


# ------------------------------------------------------------------ inputs
_TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=_DEV)


def _weights_q4k(g, rows, k):
    """Random Q4_K rows: any codes and 6-bit fields, d and dmin in [1e-4, 1e-2]."""
    w = torch.randint(0, 256, (rows, k // 256, 144), generator=g, device=_DEV, dtype=torch.uint8)
    dd = torch.rand((rows, k // 256, 2), generator=g, device=_DEV) * (1e-2 - 1e-4) + 1e-4
    w[..., 0:4] = dd.half().view(torch.uint8)
    return w.view(rows, k // 256 * 144)


def _routed(g, m, experts, topk):
    """Distinct experts per token, some experts liked more than others."""
    logits = _normal(g, m, experts) + _normal(g, experts)
    ids = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :topk]
    return ids.to(torch.int32).contiguous()


def _grouped_order(ids, groups):
    """The positions sorted by id (stable; ids below 0 in no group), and where
    each group begins."""
    flat = ids.reshape(-1).long()
    key = torch.where(flat < 0, groups, flat)
    order = torch.sort(key, stable=True).indices.to(torch.int32)
    counts = torch.bincount(key, minlength=groups + 1)[:groups]
    offsets = torch.zeros(groups + 1, dtype=torch.int32, device=_DEV)
    offsets[1:] = counts.cumsum(0).to(torch.int32)
    return offsets, order, int(counts.max())


def prepare(case, seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(int(seed) * 7919 + 17)
    s = dict(case)
    op = case["op"]
    if op == "rmsnorm":
        m, k = case["m"], case["k"]
        s["xt"] = _normal(g, m, k).to(_TYPES[case["x"]])
        s["res"] = _normal(g, m, k) * 4 if case["residual"] else None
        s["w"] = 1 + 0.1 * _normal(g, k)
        s["h"] = torch.empty((m, k), device=_DEV) if case["residual"] else None
        if case["out"] == "q8":
            s["q"] = torch.empty((m, k), dtype=torch.int8, device=_DEV)
            s["d"] = torch.empty((m, k // 32), device=_DEV)
            s["values"] = torch.empty((m, k // 32, 32), dtype=torch.float16, device=_DEV)
        else:
            s["y"] = torch.empty((m, k), dtype=_TYPES[case["out"]], device=_DEV)
    elif op == "route":
        m, experts, topk = case["m"], case["experts"], case["topk"]
        s["logits"] = _normal(g, m, experts) + _normal(g, experts)
        s["ids"] = torch.empty((m, topk), dtype=torch.int32, device=_DEV)
        s["weights"] = torch.empty((m, topk), device=_DEV)
        s["offsets"] = torch.empty(experts + 1, dtype=torch.int32, device=_DEV)
        s["order"] = torch.empty(m * topk, dtype=torch.int32, device=_DEV)
        # what grouping may need beside its outputs: far above the needed bytes
        s["ws"] = torch.empty(4 * (m * topk // 64 + 64) * (experts + 1) + 4096,
                              dtype=torch.uint8, device=_DEV)
    elif op == "combine":
        m, n, topk = case["m"], case["n"], case["topk"]
        s["y"] = _normal(g, m * topk, n)
        s["weights"] = torch.softmax(_normal(g, m, topk), dim=1)
        s["ids"] = torch.randint(0, 64, (m, topk), generator=g, device=_DEV, dtype=torch.int32)
        s["res"] = _normal(g, m, n) if case["residual"] else None
        s["out"] = torch.empty((m, n), device=_DEV)
    elif op == "grouped":
        m, experts, topk, n, k = (case[c] for c in ("m", "experts", "topk", "n", "k"))
        ids = _routed(g, m, experts, topk)
        s["offsets"], s["order"], s["most"] = _grouped_order(ids, experts)
        rows = m if case["side"] == "up" else m * topk
        x = _normal(g, rows, k)
        if case["act"] == "f16":
            s["w"] = (_normal(g, experts * n, k) * 0.05).half()
            s["x"] = x.half()
        else:
            s["w"] = _weights_q4k(g, experts * n, k)
            if case["act"] == "f32":
                s["x"] = x
            else:
                blocks = x.view(rows, k // 32, 32)
                s["d"] = blocks.abs().amax(2) / 127
                s["q"] = torch.round(blocks / s["d"][..., None]).to(torch.int8).view(rows, k)
        s["y"] = torch.empty((m * topk, n), device=_DEV)
        s["ws"] = torch.empty(m * topk * k * 8 + 65536, dtype=torch.uint8, device=_DEV)
    else:
        m, adapters, r, n, k = (case[c] for c in ("m", "adapters", "r", "n", "k"))
        # requests of uneven lengths, each with an adapter or (sometimes) none
        cuts = torch.rand(m, generator=g, device=_DEV) < max(0.02, min(1.0, 16.0 / m))
        request = torch.cumsum(cuts, 0)
        table = torch.randint(0, adapters, (m + 1,), generator=g, device=_DEV)
        table = torch.where(torch.rand(m + 1, generator=g, device=_DEV) < 0.05, -1, table)
        s["ids"] = table[request].to(torch.int32)
        s["offsets"], s["order"], _ = _grouped_order(s["ids"], adapters)
        s["xt"] = _normal(g, m, k).to(_TYPES[case["x"]])
        s["base"] = _normal(g, m, n)
        s["a"] = (_normal(g, adapters, r, k) / math.sqrt(k)).half()
        s["b"] = (_normal(g, adapters, n, r) * 0.1).half()
        ranks = torch.randint(1, r + 1, (adapters,), generator=g, device=_DEV, dtype=torch.int32)
        s["ranks"] = ranks if case["ragged"] else None
        s["scales"] = 0.5 + torch.rand(adapters, generator=g, device=_DEV)
        s["y"] = torch.zeros((m, n), device=_DEV)     # rows without an adapter stay as they are
        s["ws"] = torch.empty(m * (r + 64) * 8 + 65536, dtype=torch.uint8, device=_DEV)
    return s


# ---------------------------------------------------------------- the work
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from block_quantized_decode_q4_amd import q4k
    op = s["op"]
    if op == "rmsnorm":
        if s["out"] == "q8":
            q4k.q4k_rmsnorm(s["xt"], s["w"], s["k"], s["m"], eps=1e-5, residual=s["res"],
                            sum_out=s["h"], q=s["q"], d=s["d"])
            torch.mul(s["q"].view(s["m"], -1, 32), s["d"][..., None], out=s["values"])
            return [s["h"], s["d"], s["values"]]
        q4k.q4k_rmsnorm(s["xt"], s["w"], s["k"], s["m"], eps=1e-5, residual=s["res"],
                        sum_out=s["h"], **{"y16" if s["out"] == "f16" else "y": s["y"]})
        return [s["h"], s["y"]]
    if op == "route":
        q4k.q4k_moe_route(s["logits"], s["ids"], s["weights"], s["experts"], s["topk"], s["m"],
                          renorm=s["renorm"], offsets=s["offsets"], order=s["order"], ws=s["ws"])
        return [s["ids"], s["weights"], s["offsets"], s["order"]]
    if op == "combine":
        q4k.q4k_moe_combine(s["y"], s["weights"], s["ids"], s["out"], s["n"], s["topk"], s["m"],
                            residual=s["res"])
        return s["out"]
    if op == "grouped":
        rows = s["m"] * s["topk"]
        how = dict(x_rows=s["order"], x_div=s["topk"], x_count=s["m"])
        if s["side"] == "down":
            how = dict(y_rows=s["order"], y_count=rows)
        if s["act"] == "f16":
            q4k.q4k_f16_gemm_grouped(s["w"], s["x"], s["y"], s["offsets"], s["n"], s["k"],
                                     s["experts"], rows, **how)
        elif s["act"] == "f32":
            q4k.q4k_gemv_grouped(s["w"], s["x"], s["y"], s["offsets"], s["n"], s["k"],
                                 s["experts"], rows, ws=s["ws"], **how)
        else:
            q4k.q4k_gemv_grouped_q8(s["w"], s["q"], s["d"], s["y"], s["offsets"], s["n"], s["k"],
                                    s["experts"], rows, ws=s["ws"], **how)
        return s["y"]
    q4k.q4k_lora(s["xt"], s["a"], s["b"], s["y"], s["offsets"], s["order"], s["n"], s["k"],
                 s["r"], s["adapters"], s["m"], base=s["base"], ranks=s["ranks"],
                 scales=s["scales"], ws=s["ws"])
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


def _run_plain(s):
    op = s["op"]
    if op == "rmsnorm":
        x = s["xt"].float()
        h = x if s["res"] is None else x + s["res"]
        y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-5) * s["w"]
        shown = None if s["res"] is None else h
        if s["out"] != "q8":
            return [shown, y.to(_TYPES[s["out"]])]
        y = y.view(s["m"], -1, 32)
        top = y.abs().amax(2, keepdim=True)
        codes = torch.round(y * torch.where(top > 0, 127 / top, 0.0))
        return [shown, (top / 127)[..., 0], (codes * (top / 127)).half()]
    if op == "route":
        top = torch.sort(s["logits"], dim=1, descending=True, stable=True)
        ids, best = top.indices[:, : s["topk"]], top.values[:, : s["topk"]]
        parts = torch.exp(best - best[:, :1])
        whole = parts if s["renorm"] else torch.exp(top.values - best[:, :1])
        weights = parts / whole.sum(1, keepdim=True)
        flat = ids.reshape(-1)
        order = torch.sort(flat, stable=True)
        bounds = torch.arange(s["experts"] + 1, device=flat.device)
        offsets = torch.searchsorted(order.values, bounds)
        return [ids.int(), weights, offsets.int(), order.indices.int()]
    if op == "combine":
        out = (s["weights"][..., None] * s["y"].view(s["m"], s["topk"], s["n"])).sum(1)
        return out if s["res"] is None else out + s["res"]
    if op == "grouped":
        rows, experts, n, k = s["m"] * s["topk"], s["experts"], s["n"], s["k"]
        at = torch.arange(rows, device=_DEV)
        group = torch.searchsorted(s["offsets"], at.int(), right=True) - 1
        if s["act"] == "q8":
            x = (s["q"].view(-1, k // 32, 32) * s["d"][..., None]).view(-1, k)
        else:
            x = s["x"].float()
        x = x[s["order"] // s["topk"]] if s["side"] == "up" else x
        if rows <= experts:           # few rows: the matrices they meet, one by one
            w = s["w"].view(experts, n, -1)[group]
            w = w.float() if s["act"] == "f16" else _dequantized(w, k)
            y = torch.bmm(w, x[:, :, None])[..., 0]
        else:                         # every matrix, its rows padded to the longest group
            w = s["w"].view(experts, n, -1)
            w = w.float() if s["act"] == "f16" else _dequantized(w, k)
            place = at - s["offsets"][group]
            padded = torch.zeros((experts, s["most"], k), device=_DEV)
            padded[group, place] = x
            y = torch.bmm(w, padded.transpose(1, 2).contiguous())[group, :, place]
        if s["side"] == "up":
            return y
        out = torch.empty_like(y)
        out[s["order"].long()] = y
        return out
    m, r, adapters = s["m"], s["r"], s["adapters"]
    mine = s["ids"][:, None] == torch.arange(adapters, device=_DEV)
    keep = mine[:, :, None].float() * s["scales"][:, None]
    if s["ranks"] is not None:
        keep = keep * (torch.arange(r, device=_DEV) < s["ranks"][:, None])
    v = s["xt"].float() @ s["a"].view(adapters * r, -1).float().T
    v = v * keep.expand(m, adapters, r).reshape(m, -1)
    up = s["b"].float().permute(0, 2, 1).reshape(adapters * r, -1)
    y = s["base"] + v @ up
    return torch.where((s["ids"] >= 0)[:, None], y, 0.0)


# --------------------------------------------------- what it cannot do without
def work(case):
    op, m = case["op"], case["m"]
    if op == "rmsnorm":
        k = case["k"]
        size = {"f32": 4, "f16": 2, "bf16": 2}
        each = size[case["x"]] + (8 if case["residual"] else 0)
        each += 1.125 + 1 + 2 if case["out"] == "q8" else size[case["out"]]
        return {"bytes": m * k * each + 4 * k, "flops": 6 * m * k}
    if op == "route":
        return {"bytes": 4 * m * case["experts"] + 12 * m * case["topk"] + 4 * case["experts"],
                "flops": 4 * m * case["experts"]}
    if op == "combine":
        return {"bytes": 4 * m * case["n"] * (case["topk"] + 1 + int(case["residual"])),
                "flops": 2 * m * case["n"] * case["topk"]}
    n, k = case["n"], case["k"]
    if op == "grouped":
        experts, rows = case["experts"], m * case["topk"]
        met = experts * (1 - (1 - case["topk"] / experts) ** m)
        x_rows = m if case["side"] == "up" else rows
        w_bytes, x_bytes = {"f32": (0.5625, 4), "q8": (0.5625, 1.125), "f16": (2, 2)}[case["act"]]
        return {"bytes": met * n * k * w_bytes + x_rows * k * x_bytes + 4 * rows * n,
                "flops": 2 * rows * n * k}
    adapters, r = case["adapters"], case["r"]
    mean = (r + 1) / 2 if case["ragged"] else r
    met = adapters * (1 - (1 - 1 / adapters) ** min(m, 16))
    return {"bytes": 2 * met * mean * (n + k) + m * k * (4 if case["x"] == "f32" else 2) + 8 * m * n,
            "flops": 2 * m * mean * (n + k)}


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


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rmsnorm":
        h = s["xt"].double() + (0 if s["res"] is None else s["res"].double())
        y = h / torch.sqrt((h * h).sum(1, keepdim=True) / case["k"] + 1e-5) * s["w"].double()
        shown = None if s["res"] is None else h
        if case["out"] != "q8":
            return [shown, y]
        d = y.view(case["m"], -1, 32).abs().max(2).values / 127
        return [shown, d, torch.round(y.view(case["m"], -1, 32) / d[..., None]) * d[..., None]]
    if op == "route":
        p = torch.softmax(s["logits"].double(), dim=1)
        top = torch.sort(p, dim=1, descending=True, stable=True).values[:, : case["topk"]]
        return [None, top / top.sum(1, keepdim=True) if case["renorm"] else top, None, None]
    if op == "combine":
        out = torch.zeros((case["m"], case["n"]), dtype=torch.float64, device=_DEV)
        for j in range(case["topk"]):
            out += s["weights"][:, j: j + 1].double() * s["y"][j:: case["topk"]].double()
        return out if s["res"] is None else out + s["res"].double()
    if op == "grouped":
        n, k = case["n"], case["k"]
        begin = s["offsets"].tolist()
        order = s["order"].long()
        y = torch.empty((case["m"] * case["topk"], n), dtype=torch.float64, device=_DEV)
        for e in range(case["experts"]):
            lo, hi = begin[e], begin[e + 1]
            if lo == hi:
                continue
            at = order[lo:hi] // case["topk"] if case["side"] == "up" else slice(lo, hi)
            if case["act"] == "q8":
                x = s["q"][at].double() * s["d"][at].double().repeat_interleave(32, dim=1)
            else:
                x = s["x"][at].double()
            w = s["w"][e * n: (e + 1) * n]
            w = w.double() if case["act"] == "f16" else _exact_q4k(w, k)
            y[order[lo:hi] if case["side"] == "down" else slice(lo, hi)] = x @ w.T
        return y
    y = torch.zeros((case["m"], case["n"]), dtype=torch.float64, device=_DEV)
    for a in range(case["adapters"]):
        at = torch.nonzero(s["ids"] == a)[:, 0]
        rank = case["r"] if s["ranks"] is None else int(s["ranks"][a])
        v = s["xt"][at].double() @ s["a"][a, :rank].double().T
        y[at] = s["base"][at].double() + s["scales"][a].double() * (v @ s["b"][a, :, :rank].double().T)
    return y
