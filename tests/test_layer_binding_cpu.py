"""The binding of the operators around a layer's projections on the CPU: which
arguments reach the library.  Stand-ins take the place of GPU tensors and of
the library, so nothing is launched: a call that is let through is recorded."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from block_quantized_decode_q4_amd import q4k  # noqa: E402


class GpuTensor:
    """What the binding asks of a dense tensor on GPU 0."""

    def __init__(self, dtype, *shape):
        self.dtype, self.shape, self.device = dtype, shape, "cuda:0"

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def element_size(self):
        return torch.empty(0, dtype=self.dtype).element_size()

    def data_ptr(self):
        return 0x100000


@pytest.fixture
def calls(monkeypatch):
    """The calls that reach the library, as (name, arguments)."""
    made = []

    class Library:
        def __getattr__(self, name):
            return lambda *args: made.append((name, args)) or q4k.Q4K_OK

    q4k._import_torch()
    monkeypatch.setattr(q4k, "load_library", Library)
    monkeypatch.setattr(q4k, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(q4k, "_current_device", lambda: 0)
    return made


def _f16_grouped(w_dtype, x_dtype):
    q4k.q4k_f16_gemm_grouped(GpuTensor(w_dtype, 2 * 8, 64), GpuTensor(x_dtype, 5, 64),
                             GpuTensor(torch.float32, 5, 8), GpuTensor(torch.int32, 3), 8, 64, 2, 5)


def test_f16_grouped_takes_halves_only(calls):
    """bfloat16 is 16 bits wide too, but its bits are no binary16."""
    half = torch.float16
    for w, x in ((half, torch.bfloat16), (torch.bfloat16, half), (torch.bfloat16, torch.int16),
                 (half, torch.float32), (torch.int32, half), (torch.int8, half)):
        with pytest.raises(TypeError):
            _f16_grouped(w, x)
    assert calls == []
    for w, x in ((half, half), (torch.int16, half), (half, torch.int16), (torch.uint16, half)):
        _f16_grouped(w, x)
    assert [name for name, _ in calls] == ["q4k_f16_gemm_grouped"] * 4


def _every_call():
    """Each call with every argument that is memory: (function, its memory
    arguments by name, the rest)."""
    f32, f16, i32, u8, i8 = (torch.float32, torch.float16, torch.int32, torch.uint8, torch.int8)
    t = GpuTensor
    ws = t(u8, 1 << 16)
    rows = dict(y=t(f32, 5, 8), offsets=t(i32, 3), x_rows=t(i32, 5), y_rows=t(i32, 5))
    q4 = dict(rows, w=t(u8, 2 * 8, 144), ws=ws)
    sizes = dict(n=8, k=256, groups=2, rows=5)
    return [
        (q4k.q4k_rmsnorm, dict(x=t(f32, 2, 64), weight=t(f32, 64), residual=t(f32, 2, 64),
                               sum_out=t(f32, 2, 64), y=t(f32, 2, 64), y16=t(f16, 2, 64),
                               q=t(i8, 2, 64), d=t(f32, 2, 2)), dict(k=64, m=2)),
        (q4k.q4k_moe_route, dict(logits=t(f32, 2, 8), ids=t(i32, 2, 2), weights=t(f32, 2, 2),
                                 offsets=t(i32, 9), order=t(i32, 4), ws=ws),
         dict(n_experts=8, topk=2, m=2)),
        (q4k.q4k_moe_group, dict(ids=t(i32, 4), offsets=t(i32, 9), order=t(i32, 4), ws=ws),
         dict(count=4, groups=8)),
        (q4k.q4k_moe_combine, dict(y=t(f32, 4, 8), weights=t(f32, 2, 2), ids=t(i32, 2, 2),
                                   out=t(f32, 2, 8), residual=t(f32, 2, 8)),
         dict(n=8, topk=2, m=2)),
        (q4k.q4k_gemv_grouped, dict(q4, x=t(f32, 5, 256)), sizes),
        (q4k.q4k_gemv_grouped_q8, dict(q4, q=t(i8, 5, 256), d=t(f32, 5, 8)), sizes),
        (q4k.q4k_f16_gemm_grouped, dict(rows, w16=t(f16, 16, 256), x16=t(f16, 5, 256)), sizes),
        (q4k.q4k_lora, dict(x=t(f32, 5, 64), a=t(f16, 2, 4, 64), b=t(f16, 2, 8, 4), y=t(f32, 5, 8),
                            offsets=t(i32, 3), order=t(i32, 5), base=t(f32, 5, 8), ranks=t(i32, 2),
                            scales=t(f32, 2), ws=ws),
         dict(n=8, k=64, r=4, adapters=2, rows=5)),
    ]


def _host_array(t):
    kind = {torch.float32: np.float32, torch.float16: np.float16, torch.int32: np.int32,
            torch.uint8: np.uint8, torch.int8: np.int8}[t.dtype]
    return np.zeros(t.shape, kind)


def test_host_arrays_are_refused(calls):
    """A numpy array lies in host memory, which a kernel must not be given."""
    for call, memory, rest in _every_call():
        call(**memory, **rest)
        assert calls.pop()[0] == call.__name__
        for name, t in memory.items():
            with pytest.raises(TypeError):
                call(**dict(memory, **{name: _host_array(t)}), **rest)
            assert calls == [], (call.__name__, name)


def test_one_tensor_among_addresses(calls):
    """Addresses are taken wherever a tensor is; the one tensor left, whichever
    it is, says which device the call runs on."""
    for call, memory, rest in _every_call():
        addresses = dict.fromkeys(memory, 0x100000)
        if "ws" in memory:
            rest = dict(rest, ws_bytes=memory["ws"].numel())
        for name, t in memory.items():
            call(**dict(addresses, **{name: t}), **rest)
            assert [c[0] for c in calls] == [call.__name__], (call.__name__, name)
            calls.clear()
            host = GpuTensor(t.dtype, *t.shape)
            host.get_device = lambda: -1
            with pytest.raises(ValueError):
                call(**dict(addresses, **{name: host}), **rest)
            assert calls == [], (call.__name__, name)
