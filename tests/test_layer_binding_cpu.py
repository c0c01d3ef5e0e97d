"""The binding of the operators around a layer's projections on the CPU: which
arguments reach the library.  Stand-ins take the place of GPU tensors and of
the library, so nothing is launched: a call that is let through is recorded."""
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
