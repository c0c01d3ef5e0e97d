"""f64 definitions and tolerances of the operators at the ends of a layer's
blocks, shared by their GPU tests (torch, on the tensors' device)."""
import math

import torch

from block_quantized_decode_q4_amd import q4k

ACTS = (q4k.Q4K_ACT_NONE, q4k.Q4K_ACT_RELU, q4k.Q4K_ACT_SILU, q4k.Q4K_ACT_GELU,
        q4k.Q4K_ACT_GELU_TANH, q4k.Q4K_ACT_SIGMOID)


def act64(z, act):
    if act == q4k.Q4K_ACT_RELU:
        return torch.where(z < 0, 0.0, z)
    if act == q4k.Q4K_ACT_SILU:
        return z * torch.sigmoid(z)
    if act == q4k.Q4K_ACT_GELU:
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2))
    if act == q4k.Q4K_ACT_GELU_TANH:
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    if act == q4k.Q4K_ACT_SIGMOID:
        return torch.sigmoid(z)
    return z


def act_error(z, act):
    """The documented bound of the activation's own error at z."""
    if act in (q4k.Q4K_ACT_NONE, q4k.Q4K_ACT_RELU):
        return torch.zeros_like(z)
    a = z.abs()
    return (32 + 4 * a ** 2 + a ** 3) * 2.0 ** -24 * act64(z, act).abs() + 2.0 ** -100


def epilogue64(z, dz, act, gate, residual):
    """y and the bound of its f32 error, for a z that is off by at most dz: no
    activation is steeper than 1.13; the activation, the product and the sum are
    rounded to within half a step of 2^-23 each, one step with what their operands'
    errors add."""
    a = act64(z, act)
    g = torch.ones_like(z) if gate is None else gate.double()
    r = torch.zeros_like(z) if residual is None else residual.double()
    err = g.abs() * (1.13 * dz + act_error(z, act)) * (1 + 2.0 ** -20)
    y = a * g + r
    return y, err + 2.0 ** -23 * ((a * g).abs() + r.abs()) + 2.0 ** -126


def half_error(y, err):
    """The bound of the binary16 output: half a step (2^-11 of the value, 2^-25 near
    0) more."""
    return err * (1 + 2.0 ** -10) + 2.0 ** -11 * y.abs() + 2.0 ** -25


def assert_within(got, ref, err, what):
    got = got.double()
    bad = ~((got - ref).abs() <= err)
    if bool(bad.any()):
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError("%s: %d of %d off, first %s: %r, exact %r, bound %r" % (
            what, int(bad.sum()), bad.numel(), i, got[i].item(), ref[i].item(), err[i].item()))


def dequantized(w, k):
    """f64 weights of Q4_K rows (n x bytes, uint8), field by field."""
    sb = w.reshape(-1, 144)
    d, dmin = sb[:, 0:4].contiguous().view(torch.float16).double().unbind(1)
    s = sb[:, 4:16].long()
    out = torch.empty((sb.shape[0], 256), dtype=torch.float64, device=w.device)
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


def term_sizes(w, k):
    """|d sc q| + |dmin m| of each weight of Q4_K rows: the weights of the same rows
    with dmin's sign turned (d and dmin here are positive)."""
    t = w.reshape(-1, 144).clone()
    t[:, 3] ^= 0x80
    return dequantized(t.reshape(w.shape), k)


def random_q4k(g, rows, k, scale=0.05):
    """Q4_K rows of any codes and 6-bit fields, d and dmin positive."""
    dev = g.device
    w = torch.randint(0, 256, (rows, k // 256, 144), generator=g, device=dev, dtype=torch.uint8)
    dd = (0.1 + torch.rand((rows, k // 256, 2), generator=g, device=dev)) * (scale / math.sqrt(k))
    w[..., 0:4] = dd.half().view(torch.uint8)
    return w.view(rows, k // 256 * 144)


def norm64(v, layer, weight, bias, eps):
    if layer:
        v = v - v.mean(1, keepdim=True)
    y = v / torch.sqrt(v.square().mean(1, keepdim=True) + eps) * weight.double()
    return y if bias is None else y + bias.double()


def route64(logits, bias, sigmoid, parts, keep, topk, renorm, scale):
    """ids and weights by the definition, token by token (numpy f64)."""
    import numpy as np
    m, E = logits.shape
    each = E // parts
    ids = np.full((m, topk), -1, np.int32)
    weights = np.zeros((m, topk))
    b = np.zeros(E) if bias is None else bias.astype(np.float64)
    for t in range(m):
        l = logits[t].astype(np.float64)
        masked = np.isnan(l) | (l == -np.inf)
        with np.errstate(all="ignore"):
            if sigmoid:
                s = np.where(masked, 0.0, 1 / (1 + np.exp(-l)))
            else:
                top = l[~masked].max() if (~masked).any() else 0.0
                s = np.where(masked, 0.0, np.where(l == top, 1.0, np.exp(l - top)))
                s = s / s.sum() if s.sum() > 0 else s
            c = np.where(masked | np.isnan(b) | (b == -np.inf), -np.inf, s + b)
        if keep < parts:
            values = []
            for p in range(parts):
                best = np.sort(c[p * each: (p + 1) * each])[::-1][:2]
                best = best[best > -np.inf]
                values.append(best.sum() if len(best) else -np.inf)
            kept = [p for p in np.argsort(-np.array(values), kind="stable")[:keep]
                    if values[p] > -np.inf]
            c = np.where(np.isin(np.arange(E) // each, kept), c, -np.inf)
        chosen = [e for e in np.argsort(-c, kind="stable")[:topk] if c[e] > -np.inf]
        w = s[chosen]
        if renorm:
            w = w / w.sum() if w.sum() > 0 else w * 0
        ids[t, : len(chosen)] = chosen
        weights[t, : len(chosen)] = w * scale
    return ids, weights
