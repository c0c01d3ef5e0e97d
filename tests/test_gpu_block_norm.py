"""GPU parity of the norms on both sides of a residual's addition
(q4k_block_norm) against f64.

Sums are f64, elements f32 (steps of 2^-24 of a value, to within half of 2^-23): a
normed value carries the roundings of the factor r, of its difference from the
mean (in two steps), of the product with r and of the one with the weight, five of
them; the bias's addition, the gate's product and the residual's addition one each.
So h is within 8 2^-24 |scale gate| (|p - post_bias| + |post_bias|) + 2^-24
|residual| of the exact value, y within 6 2^-24 (|y - bias| + |bias|) of the norm of
the h that came out.  A layer norm whose mean is m times its deviation carries
2^-48 m more (the mean in two f32 numbers): below 2^-30 for means up to 2^18
deviations, held here with 1e-9 of the weight.
"""
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


TYPES = (torch.float32, torch.float16, torch.bfloat16)


def _rand(g, *shape):
    return torch.randn(shape, device="cuda", generator=g)


def _h_reference(x, layer, pw, pb, gate, scale, res, eps):
    p = x.double()
    size = p.abs()
    if pw is not None:
        p = B.norm64(p, layer, pw, None, eps)
        b = torch.zeros_like(p) if pb is None else pb.double()
        size = p.abs() + b.abs() + 1e-3 * pw.double().abs()
        p = p + b
    f = scale * (1.0 if gate is None else gate.double())
    r = torch.zeros_like(p) if res is None else res.double()
    return p * f + r, 2.0 ** -21 * size * abs(f) + 2.0 ** -24 * r.abs() + 2.0 ** -126


def _y_reference(h, layer, w, b, eps):
    y = B.norm64(h.double(), layer, w, None, eps)
    size = y.abs()
    if b is not None:
        y, size = y + b.double(), size + b.double().abs()
    return y, 6 * 2.0 ** -24 * size + 1e-9 * w.double().abs()


SHAPES = [(1, 1), (1, 7), (3, 8), (2, 9), (5, 31), (4, 64), (3, 100), (1, 513), (2, 2048), (7, 4096),
          (3, 8192), (2, 8193), (2, 8200), (1, 16384), (2, 32768), (1, 32775), (1, 40000),
          (300, 1000), (1100, 8208), (1030, 8211), (2000, 96)]


@pytest.mark.parametrize("m,k", SHAPES)
@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("post", [True, False])
def test_norms(m, k, layer, post):
    at = SHAPES.index((m, k)) + layer + 2 * post
    x_type = TYPES[at % 3]
    g = torch.Generator(device="cuda").manual_seed(at)
    x = (_rand(g, m, k) * 3 + 1).to(x_type)
    rows = (0, 1, m)[(at + layer) % 3]
    gate = _rand(g, rows, k) if rows else None
    res = _rand(g, m, k) * 4 if at % 4 else None
    pw, pb = (_rand(g, k), _rand(g, k) if at % 2 else None) if post else (None, None)
    w, b = _rand(g, k), _rand(g, k) if at % 3 == 0 else None
    scale = (1.0, 0.22, -2.5)[at % 3]
    eps = 1e-5
    h = torch.full((m, k), float("nan"), device="cuda")
    y = torch.full((m, k), float("nan"), device="cuda")
    y16 = torch.full((m, k), float("nan"), device="cuda", dtype=torch.float16)
    q = d = None
    if k % 32 == 0:
        q = torch.full((m, k), 99, device="cuda", dtype=torch.int8)
        d = torch.full((m, k // 32), float("nan"), device="cuda")
    print("block norm", m, k, x_type, "layer" if layer else "rms", post, rows, flush=True)
    kind = q4k.Q4K_NORM_LAYER if layer else q4k.Q4K_NORM_RMS
    how = dict(kind=kind, post_weight=pw, post_bias=pb, gate=gate,
               gate_stride=k if rows == m and m > 1 else 0, scale=scale, residual=res, bias=b,
               eps=eps)
    q4k.q4k_block_norm(x, w, k, m, sum_out=h, y=y, y16=y16, q=q, d=d, **how)
    ref, err = _h_reference(x, layer, pw, pb, gate, scale, res, eps)
    B.assert_within(h, ref, err, "h")
    ref, err = _y_reference(h, layer, w, b, eps)
    B.assert_within(y, ref, err, "y")
    assert torch.equal(y16, y.half())
    if q is not None:
        q_ref, d_ref = torch.empty_like(q), torch.empty_like(d)
        q4k.q4k_quantize_q8(y, q_ref, d_ref, k, m)
        assert torch.equal(q, q_ref) and torch.equal(d, d_ref)
    # without h: the same y
    again = torch.full((m, k), float("nan"), device="cuda")
    q4k.q4k_block_norm(x, w, k, m, y=again, **how)
    assert torch.equal(again, y)
    # h alone, over the residual
    if res is not None:
        over = res.clone()
        q4k.q4k_block_norm(x, None, k, m, sum_out=over, **dict(how, residual=over, bias=None))
        assert torch.equal(over, h)
        over = res.clone()
        q4k.q4k_block_norm(x, w, k, m, sum_out=over, y=again, **dict(how, residual=over))
        assert torch.equal(over, h) and torch.equal(again, y)
    if x_type is torch.float32:
        over = x.clone()
        q4k.q4k_block_norm(over, w, k, m, sum_out=over, y=again, **how)
        assert torch.equal(over, h) and torch.equal(again, y)


@pytest.mark.parametrize("m,k,pad", [(5, 64, 3), (9, 1000, 8), (3, 8193, 1)])
def test_strides(m, k, pad):
    """Rows of x and of gate apart from one another."""
    g = torch.Generator(device="cuda").manual_seed(k)
    for x_type in TYPES:
        x = torch.full((m, k + pad), float("nan"), device="cuda", dtype=x_type)
        x[:, :k] = _rand(g, m, k).to(x_type)
        gate = torch.full((m, k + 2 * pad), float("nan"), device="cuda")
        gate[:, :k] = _rand(g, m, k)
        w, pw = _rand(g, k), _rand(g, k)
        out = [torch.empty((m, k), device="cuda") for _ in range(4)]
        q4k.q4k_block_norm(x, w, k, m, x_stride=k + pad, gate=gate, gate_stride=k + 2 * pad,
                           post_weight=pw, sum_out=out[0], y=out[1])
        q4k.q4k_block_norm(x[:, :k].contiguous(), w, k, m, gate=gate[:, :k].contiguous(),
                           gate_stride=k, post_weight=pw, sum_out=out[2], y=out[3])
        assert torch.equal(out[0], out[2]) and torch.equal(out[1], out[3])


def test_far_means_and_constant_rows():
    """A layer norm of rows far from 0 keeps their deviations; a constant row
    gives its bias."""
    m, k = 4, 5000
    g = torch.Generator(device="cuda").manual_seed(1)
    x = _rand(g, m, k) + torch.tensor([[0.0], [100.0], [1000.0], [0.0]], device="cuda")
    x[3] = 12345.678
    w, b = _rand(g, k), _rand(g, k)
    y = torch.empty((m, k), device="cuda")
    q4k.q4k_block_norm(x, w, k, m, kind=q4k.Q4K_NORM_LAYER, bias=b, y=y)
    ref, err = _y_reference(x, True, w, b, 1e-5)
    B.assert_within(y, ref, err, "y")
    assert torch.equal(y[3], b)


def test_extreme_rows():
    """Squares beyond f32 and below it, zeros, infinities and NaN: each row by
    itself."""
    k = 2048
    g = torch.Generator(device="cuda").manual_seed(2)
    x = _rand(g, 7, k)
    x[1] *= 5e37
    x[2] *= 1e-41
    x[3] = 0
    x[4, 5] = float("inf")
    x[5, 9] = float("nan")
    w, pw, b = torch.ones(k, device="cuda"), _rand(g, k), _rand(g, k)
    y = torch.empty((7, k), device="cuda")
    q4k.q4k_block_norm(x, w, k, 7, y=y, bias=b, eps=0.0)
    ref, err = _y_reference(x, False, w, b, 0.0)
    for t in (0, 1, 2, 6):
        B.assert_within(y[t], ref[t], err[t], "row %d" % t)
    assert bool(y[3].isnan().all()) and bool(y[5].isnan().all())
    keep = torch.arange(k, device="cuda") != 5
    assert bool(y[4, 5].isnan()) and torch.equal(y[4, keep], b[keep])
    # through both norms: rows 4 and 5 are NaN, the others are not
    q4k.q4k_block_norm(x, w, k, 7, y=y, post_weight=pw)
    assert y.isnan().any(1).tolist() == [False, False, False, False, True, True, False]
    q4k.q4k_block_norm(x, w, k, 7, y=y, post_weight=pw, kind=q4k.Q4K_NORM_LAYER)
    assert y.isnan().all(1).tolist() == [False, False, False, False, True, True, False]


def test_past_32_bit_offsets():
    m, k = 270000, 8192
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.zeros((m, k), device="cuda", dtype=torch.float16)
    x[-2:] = _rand(g, 2, k).half()
    w = _rand(g, k)
    y16 = torch.full((m, k), float("nan"), device="cuda", dtype=torch.float16)
    q4k.q4k_block_norm(x, w, k, m, y16=y16, post_weight=w, scale=0.5)
    ref, _ = _h_reference(x[-2:], False, w, None, None, 0.5, None, 1e-5)
    ref = B.norm64(ref, False, w, None, 1e-5)
    # h's roundings, 2^-21 of it at most, move y by twice that at most; y's own are 6
    # of 2^-24
    B.assert_within(y16[-2:], ref, B.half_error(ref, 2.0 ** -19 * ref.abs() + 1e-9), "last rows")
    assert bool((y16[:-2] == 0).all())
