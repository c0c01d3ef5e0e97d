"""GPU parity of the products with an epilogue (q4k_gemv_act, q4k_f16_gemm_act,
q4k_gemv_grouped_act, q4k_f16_gemm_grouped_act) against f64.

z is off by what the product without an epilogue may be off (Q4_K: 1e-5 sum
|w||x|; grouped Q4_K: (280 + k/128) 2^-23 T + 2^-48 U, T the sum of |d sc q| +
|dmin m| times |x|, U with the row's largest |x|; fp16: k 2^-23 sum |w||x|) and
by 2^-23 |z| for the roundings of the sum and of the bias's addition; what the
epilogue adds to that is in block_ops.epilogue64.
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


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rand(g, *shape):
    return torch.randn(shape, device="cuda", generator=g)


def _i32(a):
    return torch.tensor(np.asarray(a, np.int32), device="cuda")


# what a case's epilogue has: (activation, bias, gate's type, residual, y, y16)
F32, F16 = torch.float32, torch.float16
EPILOGUES = [
    (q4k.Q4K_ACT_NONE, True, None, True, True, False),
    (q4k.Q4K_ACT_SILU, False, F32, False, True, False),
    (q4k.Q4K_ACT_GELU, True, F16, True, True, True),
    (q4k.Q4K_ACT_RELU, True, None, False, False, True),
    (q4k.Q4K_ACT_GELU_TANH, False, F16, False, False, True),
    (q4k.Q4K_ACT_SIGMOID, True, F32, True, True, True),
    (q4k.Q4K_ACT_NONE, False, None, False, True, False),
]


def _operands(g, ep, biases, shape):
    act, bias, gate, residual, y, y16 = ep
    o = dict(act=act, bias=_rand(g, *biases) if bias else None,
             gate=_rand(g, *shape).to(gate) if gate else None,
             residual=4 * _rand(g, *shape) if residual else None,
             y16=torch.full(shape, float("nan"), device="cuda", dtype=F16) if y16 else None)
    return o, torch.full(shape, float("nan"), device="cuda") if y else None


def _check(y, o, z, dz, what):
    """y and y16 of rows with sums z (bias added), off by dz."""
    dz = dz + 2.0 ** -23 * z.abs()
    ref, err = B.epilogue64(z, dz, o["act"], o["gate"], o["residual"])
    if y is not None:
        B.assert_within(y, ref, err, what)
    if o["y16"] is not None:
        B.assert_within(o["y16"], ref, B.half_error(ref, err), what + " y16")


# ---------------------------------------------------------------- Q4_K GEMV
# (n, k, m, weights 128-byte aligned, the kernel that the shape must take)
GEMVS = [(1, 256, 1, True, 2), (1001, 512, 1, True, 2), (300, 4352, 1, True, 2),
         (257, 12544, 1, True, 2), (8192, 4096, 1, True, 3), (32768, 1024, 1, True, 3),
         (9001, 4352, 1, True, 3), (2400, 14336, 1, True, 3), (33, 2048, 2, True, 4),
         (513, 4096, 2, True, 4), (64, 1024, 4, True, 5), (65, 4096, 8, True, 7),
         (1000, 256, 16, True, 5), (40000, 256, 3, True, 5), (64, 14336, 8, True, 6), (2049, 14336, 1, True, 2),
         (50, 14336, 9, True, 6), (17, 1024, 17, True, 6), (200, 768, 32, True, 6),
         (40, 512, 1, False, 2), (77, 768, 3, False, 1), (500, 4096, 8, False, 1)]


@pytest.mark.parametrize("case", GEMVS)
@pytest.mark.parametrize("which", [0, 1])
def test_gemv(case, which):
    n, k, m, aligned, kernel = case
    assert q4k.q4k_plan(n, k, m, w_aligned128=aligned).kernel == kernel
    at = GEMVS.index(case)
    ep = EPILOGUES[(2 * at + which) % len(EPILOGUES)]
    print("gemv", case, ep, flush=True)
    g = _gen(at)
    room = torch.empty(n * k // 256 * 144 + 256, dtype=torch.uint8, device="cuda")
    first = -room.data_ptr() % 128 + (0 if aligned else 16)
    w = room[first: first + n * k // 256 * 144]
    w.copy_(B.random_q4k(g, n, k).view(-1))
    x = _rand(g, m, k)
    o, y = _operands(g, ep, (n,), (m, n))
    q4k.q4k_gemv_act(w, x, y, n, k, m, **o)
    w64 = B.dequantized(w.view(n, -1), k)
    z = x.double() @ w64.T
    dz = 1e-5 * (x.double().abs() @ w64.abs().T)
    _check(y, o, z if o["bias"] is None else z + o["bias"].double(), dz, "gemv")


@pytest.mark.parametrize("n,k,m", [(300, 512, 1), (300, 4352, 1), (32768, 1024, 1), (129, 2048, 2),
                                   (40000, 256, 3), (64, 14336, 8), (200, 768, 32)])
def test_gemv_without_anything_is_the_plain_product(n, k, m):
    g = _gen(n)
    w, x = B.random_q4k(g, n, k), _rand(g, m, k)
    y = torch.empty((m, n), device="cuda")
    plain = torch.empty((m, n), device="cuda")
    q4k.q4k_gemv(w, x, plain, n, k, m)
    q4k.q4k_gemv_act(w, x, y, n, k, m)
    assert torch.equal(y, plain)


def test_gemv_whose_sums_do_not_fit_the_lds():
    """So many rows a workgroup that their sums cannot meet in LDS."""
    n, k = 3700000, 256
    plan = q4k.q4k_plan(n, k)
    assert plan.kernel == 3 and plan.lds_bytes + 8 * plan.rows_per_block > 160 * 1024
    g = _gen(3)
    w, x, res = B.random_q4k(g, n, k), _rand(g, 1, k), _rand(g, 1, n)
    y, plain = torch.empty((1, n), device="cuda"), torch.empty((1, n), device="cuda")
    q4k.q4k_gemv(w, x, plain, n, k)
    q4k.q4k_gemv_act(w, x, y, n, k, act=q4k.Q4K_ACT_RELU, residual=res)
    assert torch.equal(y, plain.clamp(min=0) + res)


# -------------------------------------------------------------- fp16 mirrors
GEMMS = [(1, 1, 64), (1, 64, 64), (2, 300, 256), (7, 33, 128), (16, 1000, 512), (63, 127, 192),
         (64, 128, 64), (65, 129, 320), (130, 257, 1024), (257, 513, 128), (509, 1000, 448),
         (300, 4096, 256), (1025, 2050, 64), (2000, 1024, 576), (33, 5000, 64), (700, 72, 2048),
         (1000, 7000, 192), (2048, 14336, 128), (1100, 9000, 320), (257, 4100, 1536), (40, 1003, 768),
         (120, 200, 64), (520, 4096, 2048)]


@pytest.mark.parametrize("m,n,k", GEMMS)
@pytest.mark.parametrize("which", [0, 1, 2])
def test_gemm(m, n, k, which):
    at = GEMMS.index((m, n, k))
    ep = EPILOGUES[(at + 2 * which) % len(EPILOGUES)]
    print("gemm", m, n, k, ep, flush=True)
    g = _gen(100 + at)
    w, x = (_rand(g, n, k) * (2 / k ** 0.5)).half(), _rand(g, m, k).half()
    o, y = _operands(g, ep, (n,), (m, n))
    q4k.q4k_f16_gemm_act(w, x, y, m, n, k, **o)
    z = x.double() @ w.double().T
    dz = k * 2.0 ** -23 * (x.double().abs() @ w.double().abs().T)
    _check(y, o, z if o["bias"] is None else z + o["bias"].double(), dz, "gemm")


# ------------------------------------------------------------------- grouped
# (rows per group, n, k, x_div): positions in a mixed order, some left out
GROUPS = [([1], 16, 256, 1), ([0, 3, 0, 1], 40, 512, 2), ([2, 1, 0, 4, 1], 1001, 256, 1),
          ([16, 17, 0, 33], 100, 768, 2), ([1] * 9, 70, 1024, 4), ([5, 0, 140], 200, 512, 1),
          ([200, 90, 1, 300], 130, 256, 2), ([0, 0], 33, 256, 1), ([3, 3], 5, 256, 1),
          ([700, 0, 900, 3], 3000, 256, 1), ([260, 129, 600], 5001, 256, 1)]


def _grouped(g, kind, sizes, n, k, x_div, ep):
    rows = sum(sizes) + 2                      # two positions in no group
    groups = len(sizes)
    rng = np.random.default_rng(rows)
    off = np.concatenate(([0], np.cumsum(sizes)))
    x_count = max(1, (rows + x_div - 1) // x_div)
    y_count = rows + 3
    x_rows = rng.permutation(rows)
    y_rows = rng.permutation(y_count)[:rows]
    if rows > 6:
        x_rows[1], y_rows[4] = -1, -5
        x_rows[2], y_rows[5] = x_count * x_div, y_count
    if kind == "q4":
        w = B.random_q4k(g, groups * n, k)
        x = _rand(g, x_count, k)
        w64, size = B.dequantized(w, k).view(groups, n, k), B.term_sizes(w, k).view(groups, n, k)
    else:
        w = (_rand(g, groups * n, k) * (2 / k ** 0.5)).half()
        x = _rand(g, x_count, k).half()
        w64 = w.double().view(groups, n, k)
        size = w64.abs()
    o, y = _operands(g, ep, (groups, n), (y_count, n))
    how = dict(x_rows=_i32(x_rows), x_div=x_div, x_count=x_count, y_rows=_i32(y_rows),
               y_count=y_count, **o)
    z = torch.full((y_count, n), float("nan"), device="cuda", dtype=torch.float64)
    dz = torch.zeros_like(z)
    for e in range(groups):
        for p in range(off[e], off[e + 1]):
            xr, yr = x_rows[p], y_rows[p]
            if xr < 0 or xr // x_div >= x_count or yr < 0 or yr >= y_count:
                continue
            v = x[xr // x_div].double()
            z[yr] = (w64[e] * v).sum(1)
            t = (size[e] * v.abs()).sum(1)
            if kind == "q4":
                dz[yr] = (280 + k / 128) * 2.0 ** -23 * t \
                    + 2.0 ** -48 * size[e].sum(1) * v.abs().max()
            else:
                dz[yr] = k * 2.0 ** -23 * t
            if o["bias"] is not None:
                z[yr] += o["bias"][e].double()
    return w, x, y, o, off, rows, how, z, dz


def _call_grouped(kind, w, x, y, off, n, k, groups, rows, how):
    if kind == "q4":
        ws = torch.full((q4k.q4k_gemv_grouped_ws(k, rows),), 0xFF, dtype=torch.uint8, device="cuda")
        q4k.q4k_gemv_grouped_act(w, x, y, _i32(off), n, k, groups, rows, ws=ws, **how)
    else:
        q4k.q4k_f16_gemm_grouped_act(w, x, y, _i32(off), n, k, groups, rows, **how)


@pytest.mark.parametrize("kind", ["q4", "f16"])
@pytest.mark.parametrize("case", GROUPS)
@pytest.mark.parametrize("which", [0, 1])
def test_grouped(kind, case, which):
    sizes, n, k, x_div = case
    at = GROUPS.index(case)
    ep = EPILOGUES[(at + 3 * which) % len(EPILOGUES)]
    print("grouped", kind, case, ep, flush=True)
    w, x, y, o, off, rows, how, z, dz = _grouped(_gen(200 + at), kind, sizes, n, k, x_div, ep)
    _call_grouped(kind, w, x, y, off, n, k, len(sizes), rows, how)
    named = ~z[:, 0].isnan()
    for out in (y, o["y16"]):
        assert out is None or bool(out[~named].isnan().all()), "rows that no position names"
    cut = {c: v if c in ("act", "bias") or v is None else v[named] for c, v in o.items()}
    _check(None if y is None else y[named], cut, z[named], dz[named], "grouped")


# ---------------------------------------------------- outputs over the operands
def _calls(g):
    """Each entry point at a shape whose last tiles overlap or are ragged: its
    output's shape and a call of it."""
    n, k, m = 300, 512, 5
    w, x = B.random_q4k(g, 2 * n, k), _rand(g, 64, k)
    w16, x16 = (_rand(g, 2 * n, k) * 0.05).half(), x.half()
    off = _i32([0, 20, 64])
    ws = torch.empty(q4k.q4k_gemv_grouped_ws(k, 64), dtype=torch.uint8, device="cuda")
    return [
        ((1, n), lambda y, **o: q4k.q4k_gemv_act(w[:n], x[:1], y, n, k, 1, **o)),
        ((m, n), lambda y, **o: q4k.q4k_gemv_act(w[:n], x[:m], y, n, k, m, **o)),
        ((64, n), lambda y, **o: q4k.q4k_f16_gemm_act(w16[:n], x16, y, 64, n, k, **o)),
        ((64, n), lambda y, **o: q4k.q4k_gemv_grouped_act(w, x, y, off, n, k, 2, 64, ws=ws, **o)),
        ((4, n), lambda y, **o: q4k.q4k_gemv_grouped_act(w, x, y, _i32([0, 3, 4]), n, k, 2, 4,
                                                         ws=ws, **o)),
        ((64, n), lambda y, **o: q4k.q4k_f16_gemm_grouped_act(w16, x16, y, off, n, k, 2, 64, **o)),
    ]


@pytest.mark.parametrize("which", range(6))
def test_in_place(which):
    """y as its own residual, y as its own gate, y16 as its own gate: the bits of
    the call with outputs apart."""
    g = _gen(5)
    shape, call = _calls(g)[which]
    a, b = _rand(g, *shape), _rand(g, *shape)
    for gate in (b, b.half()):
        apart = torch.empty(shape, device="cuda")
        half = torch.empty(shape, device="cuda", dtype=F16)
        call(apart, act=q4k.Q4K_ACT_SILU, gate=gate, residual=a, y16=half)
        y = a.clone()
        call(y, act=q4k.Q4K_ACT_SILU, gate=gate, residual=y)
        assert torch.equal(y, apart)
        over = gate.clone()
        if gate.dtype is F32:
            call(over, act=q4k.Q4K_ACT_SILU, gate=over, residual=a)
            assert torch.equal(over, apart)
        else:
            call(None, act=q4k.Q4K_ACT_SILU, gate=over, residual=a, y16=over)
            assert torch.equal(over, half)


@pytest.mark.parametrize("which", range(6))
def test_values_that_are_not_finite(which):
    """NaN and infinities in x, bias, gate and residual stay in their rows and
    columns; z = -infinity is NaN but for relu and sigmoid."""
    g = _gen(6)
    shape, call = _calls(g)[which]
    rows, n = shape
    gate, res = _rand(g, *shape), _rand(g, *shape)
    bias = torch.zeros((2, n), device="cuda")
    clean = torch.empty(shape, device="cuda")
    call(clean, act=q4k.Q4K_ACT_SILU, gate=gate, residual=res, bias=bias)
    gate[0, 1], gate[rows - 1, 2] = float("nan"), float("inf")
    res[0, 3], res[rows - 1, 4] = float("nan"), -float("inf")
    bias[:, 5], bias[:, 6] = float("nan"), -float("inf")
    y = torch.empty(shape, device="cuda")
    call(y, act=q4k.Q4K_ACT_SILU, gate=gate, residual=res, bias=bias)
    assert bool(y[0, 1].isnan()) and bool(y[0, 3].isnan()) and bool(y[:, 5:7].isnan().all())
    assert bool(y[rows - 1, 2].isinf()) and y[rows - 1, 4].item() == -float("inf")
    keep = torch.ones(shape, dtype=torch.bool, device="cuda")
    keep[0, 1] = keep[0, 3] = keep[rows - 1, 2] = keep[rows - 1, 4] = False
    keep[:, 5:7] = False
    assert torch.equal(y[keep], clean[keep])
    for act, want in ((q4k.Q4K_ACT_RELU, 0.0), (q4k.Q4K_ACT_SIGMOID, 0.0)):
        call(y, act=act, bias=bias)
        assert bool((y[:, 6] == want).all()) and bool(y[:, 5].isnan().all())


@pytest.mark.parametrize("act", B.ACTS)
def test_activations_over_their_range(act):
    """One product whose z is the bias: every size of z."""
    n, k = 4096, 64
    z = torch.cat([torch.linspace(-110, 110, 2048, device="cuda"),
                   torch.logspace(-30, 30, 1024, device="cuda"),
                   -torch.logspace(-30, 30, 1024, device="cuda")])
    w = torch.zeros((n, k), device="cuda", dtype=F16)
    x = torch.zeros((1, k), device="cuda", dtype=F16)
    y = torch.empty((1, n), device="cuda")
    q4k.q4k_f16_gemm_act(w, x, y, 1, n, k, act=act, bias=z)
    z64 = z.double()[None]
    ref = B.act64(z64, act)
    # beyond the tanh form's range its u passes f64 too: the limits
    ref = torch.where(ref.isnan(), torch.where(z64 > 0, z64, 0.0), ref)
    err = torch.nan_to_num(B.act_error(z64, act), nan=2.0 ** -100)
    small = z64.abs() > 64                     # there act is z, 0 or 1 to a step
    err = torch.where(small, 2.0 ** -22 * ref.abs() + 2.0 ** -80, err)
    B.assert_within(y, ref, err, "act %d" % act)


def test_gemm_of_rows_past_4_mi():
    """Rows so long that an operand's offsets within a tile pass 32 bits."""
    m, n, k = 2, 3, (1 << 22) + 64
    g = _gen(12)
    w, x = (_rand(g, n, k) * 2.0 ** -10).half(), _rand(g, m, k).half()
    for which in (2, 5):
        o, y = _operands(g, EPILOGUES[which], (n,), (m, n))
        q4k.q4k_f16_gemm_act(w, x, y, m, n, k, **o)
        z = x.double() @ w.double().T + o["bias"].double()
        _check(y, o, z, k * 2.0 ** -23 * (x.double().abs() @ w.double().abs().T), "long rows")


def test_grouped_x_of_4_gib():
    """x rows whose offsets pass 32 bits."""
    n, k, groups, rows = 96, 4096, 2, 130
    x_count = (1 << 31) // k + 3
    g = _gen(13)
    w = (_rand(g, groups * n, k) * 0.03).half()
    x = torch.zeros((x_count, k), device="cuda", dtype=F16)
    x[:8], x[-8:] = _rand(g, 8, k).half(), _rand(g, 8, k).half()
    x_rows = np.concatenate([np.arange(8), x_count - 1 - np.arange(8)])[np.arange(rows) % 16]
    off = [0, 50, rows]
    o, y = _operands(g, EPILOGUES[2], (groups, n), (rows, n))
    q4k.q4k_f16_gemm_grouped_act(w, x, y, _i32(off), n, k, groups, rows, x_rows=_i32(x_rows),
                                 x_count=x_count, **o)
    z = torch.empty((rows, n), device="cuda", dtype=torch.float64)
    dz = torch.empty_like(z)
    xs = x[torch.from_numpy(x_rows).cuda()].double()
    for e in range(groups):
        at = slice(off[e], off[e + 1])
        w64 = w[e * n: (e + 1) * n].double()
        z[at] = xs[at] @ w64.T + o["bias"][e].double()
        dz[at] = k * 2.0 ** -23 * (xs[at].abs() @ w64.abs().T)
    _check(y, o, z, dz, "grouped")


def test_gemm_past_32_bit_offsets():
    """2.2e9 outputs, gates and residuals: the last rows."""
    m, n, k = 70000, 32001, 64
    g = _gen(9)
    w, x = (_rand(g, n, k) * 0.25).half(), _rand(g, m, k).half()
    gate = torch.zeros((m, n), device="cuda", dtype=F16)
    y16 = torch.full((m, n), float("nan"), device="cuda", dtype=F16)
    last = slice(m - 3, m)
    gate[last] = _rand(g, 3, n).half()
    q4k.q4k_f16_gemm_act(w, x, None, m, n, k, gate=gate, y16=y16, act=q4k.Q4K_ACT_GELU)
    z = x[last].double() @ w.double().T
    dz = k * 2.0 ** -23 * (x[last].double().abs() @ w.double().abs().T)
    o = dict(act=q4k.Q4K_ACT_GELU, gate=gate[last], residual=None, y16=y16[last])
    _check(None, o, z, dz, "last rows")
    assert bool((y16[: m - 3] == 0).all())
