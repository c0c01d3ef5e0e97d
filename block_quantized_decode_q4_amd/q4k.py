"""Thin ctypes binding of libq4k.so (C ABI in include/q4k.h).

Argument marshalling only: every step of the GEMV runs in the HIP kernels of
libq4k.so.  Arguments may be torch tensors (their data_ptr() is passed) or
plain integers holding device addresses.  ``stream`` defaults to torch's
current HIP stream.  A non-zero status raises Q4KError.  If libq4k.so has not
been built, loading raises immediately -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libq4k.so")

Q4K_OK = 0
Q4K_ERR_NULL = 1
Q4K_ERR_SHAPE = 2
Q4K_ERR_SIZE = 3
Q4K_ERR_ALIGN = 4
Q4K_ERR_UNSUPPORTED = 5
Q4K_ERR_HIP = 1000

Q4K_F32 = 0
Q4K_F16 = 1
Q4K_BF16 = 2

# every symbol include/q4k.h declares
EXPORTED = (
    "q4k_row_bytes",
    "q4k_load",
    "q4k_gemv",
    "q4k_dequantize",
    "q4k_status_string",
    "q4k_gemv_ex",
    "q4k_read_calibrate",
    "q4k_read_calibrate_blocks",
    "q4k_plan",
    "q4k_gemv_q8",
    "q4k_quantize_q8",
    "q6k_row_bytes",
    "q6k_load",
    "q6k_gemv",
    "q6k_gemv_ex",
    "q6k_plan",
    "q6k_dequantize",
    "q4k_mirror_f16",
    "q6k_mirror_f16",
    "q4k_f16_cvt",
    "q4k_f16_gemm",
    "q4k_f16_gemm_f32x",
    "q4k_f16_gemm_f32x_noalloc",
    "q4k_rmsnorm",
    "q4k_moe_group_ws",
    "q4k_moe_route",
    "q4k_moe_group",
    "q4k_moe_combine",
    "q4k_gemv_grouped_ws",
    "q4k_gemv_grouped",
    "q4k_gemv_grouped_q8",
    "q4k_f16_gemm_grouped",
    "q4k_lora_ws",
    "q4k_lora",
)


class Q4KError(RuntimeError):
    def __init__(self, rc: int, where: str):
        self.rc = rc
        super().__init__("%s failed: status %d (%s)" % (where, rc, status_string(rc)))


class q4k_launch(ctypes.Structure):
    _fields_ = [
        ("variant", ctypes.c_int32),
        ("spans_per_chunk", ctypes.c_int32),
        ("rows_per_block", ctypes.c_int32),
        ("rows_per_wave", ctypes.c_int32),
        ("waves_per_block", ctypes.c_int32),
        ("x_in_registers", ctypes.c_int32),
        ("kernel", ctypes.c_int32),
        ("ring_depth", ctypes.c_int32),
        ("rows_per_task", ctypes.c_int32),
        ("cols_per_task", ctypes.c_int32),
    ]


class q4k_plan_info(ctypes.Structure):
    _fields_ = [
        ("kernel", ctypes.c_int32),
        ("grid", ctypes.c_int32),
        ("threads", ctypes.c_int32),
        ("lds_bytes", ctypes.c_int32),
        ("rows_per_block", ctypes.c_int32),
        ("cols_per_task", ctypes.c_int32),
        ("ring_depth", ctypes.c_int32),
        ("spans_per_chunk", ctypes.c_int32),
    ]


class q6k_launch(ctypes.Structure):
    _fields_ = [
        ("unit_bytes", ctypes.c_int32),
        ("batch_bytes", ctypes.c_int32),
        ("waves_per_block", ctypes.c_int32),
        ("column_groups", ctypes.c_int32),
        ("tiles_per_block", ctypes.c_int32),
    ]


class q6k_plan_info(ctypes.Structure):
    _fields_ = [
        ("unit_bytes", ctypes.c_int32),
        ("batch_bytes", ctypes.c_int32),
        ("waves_per_block", ctypes.c_int32),
        ("column_groups", ctypes.c_int32),
        ("rows_per_block", ctypes.c_int32),
        ("grid", ctypes.c_int32),
        ("lds_bytes", ctypes.c_int32),
    ]


VARIANT_AUTO = 0
VARIANT_SINGLE = 1
VARIANT_CHUNKED = 2

_lock = threading.Lock()
_lib = None


def load_library():
    """Load libq4k.so (raises OSError/RuntimeError when it is missing)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libq4k.so is not built (%s); run "
                               "`python -m block_quantized_decode_q4_amd.build`" % LIB_PATH)
        lib = ctypes.CDLL(LIB_PATH)
        vp = ctypes.c_void_p
        i64 = ctypes.c_int64
        lib.q4k_row_bytes.argtypes = [i64]
        lib.q4k_row_bytes.restype = ctypes.c_size_t
        lib.q4k_load.argtypes = [vp, vp, ctypes.c_size_t, i64, i64, vp]
        lib.q4k_load.restype = ctypes.c_int
        lib.q4k_gemv.argtypes = [vp, vp, vp, i64, i64, i64, vp]
        lib.q4k_gemv.restype = ctypes.c_int
        lib.q4k_gemv_ex.argtypes = [vp, vp, vp, i64, i64, i64, ctypes.POINTER(q4k_launch), vp]
        lib.q4k_gemv_ex.restype = ctypes.c_int
        lib.q4k_dequantize.argtypes = [vp, vp, i64, i64, vp]
        lib.q4k_dequantize.restype = ctypes.c_int
        lib.q4k_gemv_q8.argtypes = [vp, vp, vp, i64, i64, i64, vp]
        lib.q4k_gemv_q8.restype = ctypes.c_int
        lib.q4k_quantize_q8.argtypes = [vp, vp, vp, i64, i64, vp]
        lib.q4k_quantize_q8.restype = ctypes.c_int
        lib.q6k_row_bytes.argtypes = [i64]
        lib.q6k_row_bytes.restype = ctypes.c_size_t
        lib.q6k_load.argtypes = [vp, vp, ctypes.c_size_t, i64, i64, i64, vp]
        lib.q6k_load.restype = ctypes.c_int
        lib.q6k_gemv.argtypes = [vp, vp, vp, i64, i64, i64, vp]
        lib.q6k_gemv.restype = ctypes.c_int
        lib.q6k_gemv_ex.argtypes = [vp, vp, vp, i64, i64, i64, ctypes.POINTER(q6k_launch), vp]
        lib.q6k_gemv_ex.restype = ctypes.c_int
        lib.q6k_plan.argtypes = [i64, i64, i64, ctypes.c_int, ctypes.POINTER(q6k_launch),
                                 ctypes.c_size_t, ctypes.POINTER(q6k_plan_info)]
        lib.q6k_plan.restype = ctypes.c_int
        lib.q6k_dequantize.argtypes = [vp, vp, i64, i64, i64, vp]
        lib.q6k_dequantize.restype = ctypes.c_int
        lib.q4k_mirror_f16.argtypes = [vp, vp, i64, i64, vp]
        lib.q4k_mirror_f16.restype = ctypes.c_int
        lib.q6k_mirror_f16.argtypes = [vp, vp, i64, i64, i64, vp]
        lib.q6k_mirror_f16.restype = ctypes.c_int
        lib.q4k_f16_cvt.argtypes = [vp, vp, i64, vp]
        lib.q4k_f16_cvt.restype = ctypes.c_int
        lib.q4k_f16_gemm.argtypes = [vp, vp, vp, i64, i64, i64, vp]
        lib.q4k_f16_gemm.restype = ctypes.c_int
        lib.q4k_f16_gemm_f32x.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp]
        lib.q4k_f16_gemm_f32x.restype = ctypes.c_int
        lib.q4k_f16_gemm_f32x_noalloc.argtypes = [vp, vp, vp, i64, i64, i64, vp]
        lib.q4k_f16_gemm_f32x_noalloc.restype = ctypes.c_int
        lib.q4k_status_string.argtypes = [ctypes.c_int]
        lib.q4k_status_string.restype = ctypes.c_char_p
        lib.q4k_read_calibrate.argtypes = [vp, ctypes.c_size_t, vp, vp]
        lib.q4k_read_calibrate.restype = ctypes.c_int
        lib.q4k_read_calibrate_blocks.argtypes = []
        lib.q4k_read_calibrate_blocks.restype = ctypes.c_int
        lib.q4k_plan.argtypes = [i64, i64, i64, ctypes.POINTER(q4k_launch), ctypes.c_int,
                                 ctypes.c_size_t, ctypes.POINTER(q4k_plan_info)]
        lib.q4k_plan.restype = ctypes.c_int
        ci = ctypes.c_int
        sz = ctypes.c_size_t
        grouped = [vp, vp, vp, i64, i64, i64, i64, i64, i64, i64]   # offsets .. y_count
        for name, args, res in (
                ("q4k_rmsnorm", [vp, ci, i64, vp, vp, vp, vp, vp, vp, vp, i64, i64,
                                 ctypes.c_float, vp], ci),
                ("q4k_moe_group_ws", [i64, i64, i64], sz),
                ("q4k_moe_route", [vp, i64, vp, vp, vp, vp, i64, i64, ci, i64, vp, sz, vp], ci),
                ("q4k_moe_group", [vp, vp, vp, i64, i64, vp, sz, vp], ci),
                ("q4k_moe_combine", [vp, vp, vp, vp, vp, i64, i64, i64, vp], ci),
                ("q4k_gemv_grouped_ws", [i64, i64], sz),
                ("q4k_gemv_grouped", [vp, vp, vp] + grouped + [vp, sz, vp], ci),
                ("q4k_gemv_grouped_q8", [vp, vp, vp, vp] + grouped + [vp, sz, vp], ci),
                ("q4k_f16_gemm_grouped", [vp, vp, vp] + grouped + [vp], ci),
                ("q4k_lora_ws", [i64, i64], sz),
                ("q4k_lora", [vp, ci, vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, vp,
                              sz, vp], ci)):
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        _lib = lib
        return lib


def _addr(a):
    """Device/host address of a torch tensor, numpy array or int (0 for None)."""
    if a is None:
        return None
    if isinstance(a, int):
        return a
    if hasattr(a, "data_ptr"):
        if not a.is_contiguous():
            raise ValueError("tensor must be contiguous")
        return a.data_ptr()
    if hasattr(a, "ctypes"):
        return a.ctypes.data
    raise TypeError("expected a tensor, an array or an integer address, got %r" % type(a))


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc: int, where: str) -> None:
    if rc != Q4K_OK:
        raise Q4KError(rc, where)


def status_string(rc: int) -> str:
    return load_library().q4k_status_string(int(rc)).decode()


q4k_status_string = status_string


def q4k_row_bytes(k: int) -> int:
    return int(load_library().q4k_row_bytes(int(k)))


def q4k_load(w_dev, src_host, n: int, k: int, stream=None, src_bytes: int | None = None) -> None:
    """Copy Q4_K bytes from host memory into the device buffer w_dev
    (synchronous on stream)."""
    if src_bytes is None:
        src_bytes = src_host.nbytes if hasattr(src_host, "nbytes") else len(src_host)
    _check(load_library().q4k_load(_addr(w_dev), _addr(src_host), int(src_bytes), int(n), int(k),
                                   _stream(stream)), "q4k_load")


def q4k_gemv(w, x, y, n: int, k: int, m: int = 1, stream=None) -> None:
    """y[b*n + r] = sum_c W[r][c] x[b*k + c]; asynchronous on stream."""
    _check(load_library().q4k_gemv(_addr(w), _addr(x), _addr(y), int(n), int(k), int(m),
                                   _stream(stream)), "q4k_gemv")


def q4k_gemv_ex(w, x, y, n: int, k: int, m: int = 1, stream=None, **opts) -> None:
    """q4k_gemv with explicit launch options (fields of q4k_launch)."""
    cfg = q4k_launch(**{f: int(opts.get(f, 0)) for f, _ in q4k_launch._fields_})
    unknown = set(opts) - {f for f, _ in q4k_launch._fields_}
    if unknown:
        raise TypeError("unknown launch options %s" % sorted(unknown))
    _check(load_library().q4k_gemv_ex(_addr(w), _addr(x), _addr(y), int(n), int(k), int(m),
                                      ctypes.byref(cfg), _stream(stream)), "q4k_gemv_ex")


def q4k_dequantize(w, out, n: int, k: int, stream=None) -> None:
    """out[r*k + c] = W[r][c] in f32 (bit-exact); asynchronous on stream."""
    _check(load_library().q4k_dequantize(_addr(w), _addr(out), int(n), int(k), _stream(stream)),
           "q4k_dequantize")


def q4k_gemv_q8(w, x, y, n: int, k: int, m: int = 1, stream=None) -> None:
    """y = W x with x quantized to Q8 inside the kernel (the integer-dot
    variant, its own tolerance: see include/q4k.h); asynchronous."""
    _check(load_library().q4k_gemv_q8(_addr(w), _addr(x), _addr(y), int(n), int(k), int(m),
                                      _stream(stream)), "q4k_gemv_q8")


def q4k_quantize_q8(x, q, d, k: int, m: int = 1, stream=None) -> None:
    """The Q8 codes (int8, m x k) and scales (f32, m x k/32) of x (f32, m x k)
    that q4k_gemv_q8 uses; asynchronous."""
    _check(load_library().q4k_quantize_q8(_addr(x), _addr(q), _addr(d), int(k), int(m),
                                          _stream(stream)), "q4k_quantize_q8")


def q4k_plan(n: int, k: int, m: int = 1, w_aligned128: bool = True, lds_max: int = 0,
             **opts) -> q4k_plan_info:
    """The launch q4k_gemv_ex would make (no launch).  lds_max = 0 asks the
    current device; a nonzero value needs no GPU."""
    cfg = q4k_launch(**opts) if opts else None
    out = q4k_plan_info()
    _check(load_library().q4k_plan(int(n), int(k), int(m), ctypes.byref(cfg) if cfg else None,
                                   1 if w_aligned128 else 0, int(lds_max), ctypes.byref(out)),
           "q4k_plan")
    return out


def q6k_row_bytes(k: int) -> int:
    return int(load_library().q6k_row_bytes(int(k)))


def q6k_load(w_dev, src_host, n: int, k: int, row_stride: int = 0, stream=None,
             src_bytes: int | None = None) -> None:
    """Copy dense Q6_K rows from host memory into w_dev at row_stride
    (synchronous on stream)."""
    if src_bytes is None:
        src_bytes = src_host.nbytes if hasattr(src_host, "nbytes") else len(src_host)
    _check(load_library().q6k_load(_addr(w_dev), _addr(src_host), int(src_bytes), int(n), int(k),
                                   int(row_stride), _stream(stream)), "q6k_load")


def q6k_gemv(w, x, y, n: int, k: int, row_stride: int = 0, stream=None) -> None:
    """y[r] = sum_c W[r][c] x[c] over Q6_K rows; asynchronous on stream."""
    _check(load_library().q6k_gemv(_addr(w), _addr(x), _addr(y), int(n), int(k), int(row_stride),
                                   _stream(stream)), "q6k_gemv")


def q6k_gemv_ex(w, x, y, n: int, k: int, row_stride: int = 0, stream=None, **opts) -> None:
    """q6k_gemv with explicit launch options (fields of q6k_launch)."""
    unknown = set(opts) - {f for f, _ in q6k_launch._fields_}
    if unknown:
        raise TypeError("unknown launch options %s" % sorted(unknown))
    cfg = q6k_launch(**{f: int(opts.get(f, 0)) for f, _ in q6k_launch._fields_})
    _check(load_library().q6k_gemv_ex(_addr(w), _addr(x), _addr(y), int(n), int(k),
                                      int(row_stride), ctypes.byref(cfg), _stream(stream)),
           "q6k_gemv_ex")


def q6k_plan(n: int, k: int, row_stride: int = 0, w_aligned128: bool = True, lds_max: int = 0,
             **opts) -> q6k_plan_info:
    """The launch q6k_gemv_ex would make (no launch); lds_max = 0 asks the
    current device, a nonzero value needs no GPU."""
    cfg = q6k_launch(**opts) if opts else None
    out = q6k_plan_info()
    _check(load_library().q6k_plan(int(n), int(k), int(row_stride), 1 if w_aligned128 else 0,
                                   ctypes.byref(cfg) if cfg else None, int(lds_max),
                                   ctypes.byref(out)), "q6k_plan")
    return out


def q6k_dequantize(w, out, n: int, k: int, row_stride: int = 0, stream=None) -> None:
    """out[r*k + c] = W[r][c] in f32 (bit-exact); asynchronous on stream."""
    _check(load_library().q6k_dequantize(_addr(w), _addr(out), int(n), int(k), int(row_stride),
                                         _stream(stream)), "q6k_dequantize")


def q4k_mirror_f16(w, w16, n: int, k: int, stream=None) -> None:
    """The fp16 mirror (n x k halves) of dense Q4_K rows; asynchronous."""
    _check(load_library().q4k_mirror_f16(_addr(w), _addr(w16), int(n), int(k), _stream(stream)),
           "q4k_mirror_f16")


def q6k_mirror_f16(w, w16, n: int, k: int, row_stride: int = 0, stream=None) -> None:
    """The fp16 mirror (n x k halves) of Q6_K rows; asynchronous."""
    _check(load_library().q6k_mirror_f16(_addr(w), _addr(w16), int(n), int(k), int(row_stride),
                                         _stream(stream)), "q6k_mirror_f16")


def q4k_f16_cvt(x, x16, count: int, stream=None) -> None:
    """x16 = binary16 of x (nearest even); asynchronous."""
    _check(load_library().q4k_f16_cvt(_addr(x), _addr(x16), int(count), _stream(stream)),
           "q4k_f16_cvt")


def q4k_f16_gemm(w16, x16, y, m: int, n: int, k: int, stream=None) -> None:
    """y (m x n, f32) = x16 (m x k) @ w16 (n x k)^T on the matrix cores."""
    _check(load_library().q4k_f16_gemm(_addr(w16), _addr(x16), _addr(y), int(m), int(n), int(k),
                                       _stream(stream)), "q4k_f16_gemm")


def q4k_f16_gemm_f32x(w16, x, xh, y, m: int, n: int, k: int, stream=None) -> None:
    """Convert x (f32, m x k) into the scratch xh, then q4k_f16_gemm."""
    _check(load_library().q4k_f16_gemm_f32x(_addr(w16), _addr(x), _addr(xh), _addr(y), int(m),
                                            int(n), int(k), _stream(stream)),
           "q4k_f16_gemm_f32x")


def q4k_f16_gemm_f32x_noalloc(w16, x, y, m: int, n: int, k: int, stream=None) -> None:
    """q4k_f16_gemm_f32x with the library's static scratch (m*k <= 4 Mi);
    calls on one GPU must not overlap."""
    _check(load_library().q4k_f16_gemm_f32x_noalloc(_addr(w16), _addr(x), _addr(y), int(m),
                                                    int(n), int(k), _stream(stream)),
           "q4k_f16_gemm_f32x_noalloc")


# ---------------------------------------- around a layer's projections
# These run where their tensors live: the device of the first tensor, made
# current for the call when it is not, on that device's current stream unless
# one is given.  A tensor on another device, of another type than the call
# takes, not dense or too short is refused before the call, and so is any
# object but a tensor or an integer address (an array in host memory).
_torch = None
_raw_stream = None          # device index -> address of its current stream
_current_device = None


def _import_torch():
    global _torch, _raw_stream, _current_device
    import torch
    # the calls behind torch.cuda.current_stream and current_device, without the
    # objects around them (about 1.5 us of a call); the public ones where a
    # torch has them no more
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda i: torch.cuda.current_stream(i).cuda_stream)
    _current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    _torch = torch


def _device(*args):
    """Index of the device of the first tensor among args (None: no tensor)."""
    if _torch is None:
        _import_torch()
    for a in args:
        if hasattr(a, "get_device"):
            index = a.get_device()
            if index < 0:
                raise ValueError("expected a tensor on the GPU, got one on %s" % a.device)
            return index
    return None


def _at(a, dtype, count, dev):
    """Address of a (None and integer addresses as they are); a tensor is
    dense, on device dev, of type dtype (None: any) and holds at least count
    elements."""
    if a is None or type(a) is int:
        return a
    if not hasattr(a, "get_device"):
        if isinstance(a, int):
            return int(a)
        raise TypeError("expected a tensor on the GPU or its address, got %s" % type(a))
    if a.get_device() != dev:
        raise ValueError("tensors on more than one device: %s and cuda:%s" % (a.device, dev))
    if a.dtype is not dtype and dtype is not None:
        raise TypeError("expected %s, got %s" % (dtype, a.dtype))
    if not a.is_contiguous():
        raise ValueError("tensor must be contiguous")
    if a.numel() < count:
        raise ValueError("a tensor of %d elements where %d are needed" % (a.numel(), count))
    return a.data_ptr()


def _rows_at(a, dtype, rows, width, stride, dev):
    """Address of rows of width elements, stride apart (0: dense); a tensor may
    be a view that skips the rest of each row."""
    if not stride or not hasattr(a, "get_device") or a.is_contiguous():
        return _at(a, dtype, (rows - 1) * (stride or width) + width, dev)
    if a.get_device() != dev:
        raise ValueError("tensors on more than one device: %s and cuda:%s" % (a.device, dev))
    if a.dtype is not dtype and dtype is not None:
        raise TypeError("expected %s, got %s" % (dtype, a.dtype))
    want = stride
    fits = a.dim() > 1 and a.stride(-1) == 1 and a.shape[-1] >= width
    for i in range(a.dim() - 2, -1, -1):
        fits = fits and (a.shape[i] == 1 or a.stride(i) == want)
        want *= a.shape[i]
    if not fits or want < rows * stride:
        raise ValueError("%d rows of %d elements, %d apart, in a tensor of shape %s and strides %s"
                         % (rows, width, stride, tuple(a.shape), a.stride()))
    return a.data_ptr()


def _run(fn, where, dev, stream, *args):
    """fn(*args, stream) with device dev current; raises for its status."""
    if dev is None:
        rc = fn(*args, _stream(stream))
    else:
        if stream is None:
            stream = _raw_stream(dev)
        elif not isinstance(stream, int):
            stream = stream.cuda_stream
        if dev == _current_device():
            rc = fn(*args, stream)
        else:
            with _torch.cuda.device(dev):
                rc = fn(*args, stream)
    if rc != Q4K_OK:
        raise Q4KError(rc, where)


def _act_type(x, x_type):
    """The q4k_type of x: its tensor's, or given beside an address."""
    if not hasattr(x, "get_device"):
        return Q4K_F32 if x_type is None else int(x_type)
    dtype = x.dtype
    if dtype is _torch.float32:
        have = Q4K_F32
    elif dtype is _torch.float16:
        have = Q4K_F16
    elif dtype is _torch.bfloat16:
        have = Q4K_BF16
    else:
        raise TypeError("expected f32, f16 or bf16 activations, got %s" % dtype)
    if x_type is not None and x_type != have:
        raise TypeError("x_type %s for activations of type %s" % (x_type, dtype))
    return have


def _ws_bytes(ws, ws_bytes):
    """Bytes of ws: its tensor's, or given beside an address."""
    if not hasattr(ws, "element_size"):
        return 0 if ws_bytes is None else int(ws_bytes)
    have = ws.numel() * ws.element_size()
    if ws_bytes is not None and ws_bytes > have:
        raise ValueError("a workspace of %d bytes where %d are given" % (have, ws_bytes))
    return have if ws_bytes is None else int(ws_bytes)


def q4k_rmsnorm(x, weight, k: int, m: int = 1, *, eps: float = 1e-5, residual=None, sum_out=None,
                y=None, y16=None, q=None, d=None, x_stride: int = 0, x_type=None,
                stream=None) -> None:
    """h = x + residual, y = h * weight / sqrt(mean h^2 + eps) for m rows of
    k: h to sum_out, y to any of y (f32), y16 (f16) and q, d (Q8 codes and
    scales); x f32, f16 or bf16, its rows x_stride elements apart (0: k);
    asynchronous on stream."""
    dev = _device(x, weight, residual, sum_out, y, y16, q, d)
    mk = m * k
    f32, i8, f16 = _torch.float32, _torch.int8, _torch.float16
    _run(load_library().q4k_rmsnorm, "q4k_rmsnorm", dev, stream,
         _rows_at(x, None, m, k, x_stride, dev), _act_type(x, x_type), int(x_stride),
         _at(residual, f32, mk, dev), _at(weight, f32, k, dev), _at(sum_out, f32, mk, dev),
         _at(y, f32, mk, dev), _at(y16, f16, mk, dev), _at(q, i8, mk, dev),
         _at(d, f32, mk // 32, dev), int(k), int(m), float(eps))


def q4k_moe_group_ws(slots: int, groups: int, topk: int = 1) -> int:
    """Bytes of workspace of q4k_moe_group and q4k_moe_route."""
    return int(load_library().q4k_moe_group_ws(int(slots), int(groups), int(topk)))


def q4k_moe_route(logits, ids, weights, n_experts: int, topk: int, m: int = 1, *,
                  renorm: bool = True, offsets=None, order=None, ws=None, ws_bytes=None,
                  logits_stride: int = 0, stream=None) -> None:
    """The topk experts of m tokens (ids, softmax weights) and, with offsets
    and order, their slots grouped by expert; asynchronous on stream."""
    dev = _device(logits, ids, weights, offsets, order, ws)
    f32, i32 = _torch.float32, _torch.int32
    slots = m * topk
    _run(load_library().q4k_moe_route, "q4k_moe_route", dev, stream,
         _rows_at(logits, f32, m, n_experts, logits_stride, dev), int(logits_stride),
         _at(ids, i32, slots, dev), _at(weights, f32, slots, dev), _at(offsets, i32, n_experts + 1, dev),
         _at(order, i32, slots, dev), int(n_experts), int(topk), 1 if renorm else 0, int(m),
         _at(ws, None, 0, dev), _ws_bytes(ws, ws_bytes))


def q4k_moe_group(ids, offsets, order, count: int, groups: int, *, ws=None, ws_bytes=None,
                  stream=None) -> None:
    """Slots grouped by id (order), and where each group begins (offsets);
    asynchronous on stream."""
    dev = _device(ids, offsets, order, ws)
    i32 = _torch.int32
    _run(load_library().q4k_moe_group, "q4k_moe_group", dev, stream, _at(ids, i32, count, dev),
         _at(offsets, i32, groups + 1, dev), _at(order, i32, count, dev), int(count),
         int(groups), _at(ws, None, 0, dev), _ws_bytes(ws, ws_bytes))


def q4k_moe_combine(y, weights, ids, out, n: int, topk: int, m: int = 1, *, residual=None,
                    stream=None) -> None:
    """out[t] = residual[t] + sum_j weights[t][j] y[t * topk + j] over the
    choices with an id (ids None: all); asynchronous on stream."""
    dev = _device(y, weights, ids, out, residual)
    f32 = _torch.float32
    mt = m * topk
    _run(load_library().q4k_moe_combine, "q4k_moe_combine", dev, stream, _at(y, f32, mt * n, dev),
         _at(weights, f32, mt, dev), _at(ids, _torch.int32, mt, dev),
         _at(residual, f32, m * n, dev), _at(out, f32, m * n, dev), int(n), int(topk),
         int(m))


def q4k_gemv_grouped_ws(k: int, rows: int) -> int:
    """Bytes of workspace of q4k_gemv_grouped and q4k_gemv_grouped_q8."""
    return int(load_library().q4k_gemv_grouped_ws(int(k), int(rows)))


def q4k_gemv_grouped(w, x, y, offsets, n: int, k: int, groups: int, rows: int, *, x_rows=None,
                     x_div: int = 1, x_count=None, y_rows=None, y_count=None, ws=None,
                     ws_bytes=None, stream=None) -> None:
    """Position p of group g: y[y_rows[p]] = W_g x[x_rows[p] // x_div], W_g
    in Q4_K, x f32 (counts default to rows); asynchronous on stream."""
    dev = _device(w, x, y, offsets, x_rows, y_rows, ws)
    f32, i32 = _torch.float32, _torch.int32
    x_count = rows if x_count is None else x_count
    y_count = rows if y_count is None else y_count
    _run(load_library().q4k_gemv_grouped, "q4k_gemv_grouped", dev, stream,
         _at(w, _torch.uint8, groups * n * (k // 256) * 144, dev), _at(x, f32, x_count * k, dev),
         _at(y, f32, y_count * n, dev), _at(offsets, i32, groups + 1, dev),
         _at(x_rows, i32, rows, dev), _at(y_rows, i32, rows, dev), int(n), int(k), int(groups),
         int(rows), int(x_div), int(x_count), int(y_count), _at(ws, None, 0, dev),
         _ws_bytes(ws, ws_bytes))


def q4k_gemv_grouped_q8(w, q, d, y, offsets, n: int, k: int, groups: int, rows: int, *,
                        x_rows=None, x_div: int = 1, x_count=None, y_rows=None, y_count=None,
                        ws=None, ws_bytes=None, stream=None) -> None:
    """q4k_gemv_grouped with x in Q8: codes q (int8) and scales d (f32, one
    per 32); asynchronous on stream."""
    dev = _device(w, q, d, y, offsets, x_rows, y_rows, ws)
    f32, i32 = _torch.float32, _torch.int32
    x_count = rows if x_count is None else x_count
    y_count = rows if y_count is None else y_count
    _run(load_library().q4k_gemv_grouped_q8, "q4k_gemv_grouped_q8", dev, stream,
         _at(w, _torch.uint8, groups * n * (k // 256) * 144, dev),
         _at(q, _torch.int8, x_count * k, dev), _at(d, f32, x_count * (k // 32), dev),
         _at(y, f32, y_count * n, dev), _at(offsets, i32, groups + 1, dev),
         _at(x_rows, i32, rows, dev), _at(y_rows, i32, rows, dev), int(n), int(k), int(groups),
         int(rows), int(x_div), int(x_count), int(y_count), _at(ws, None, 0, dev),
         _ws_bytes(ws, ws_bytes))


def q4k_f16_gemm_grouped(w16, x16, y, offsets, n: int, k: int, groups: int, rows: int, *,
                         x_rows=None, x_div: int = 1, x_count=None, y_rows=None, y_count=None,
                         stream=None) -> None:
    """q4k_gemv_grouped on fp16 mirrors (groups * n x k halves) and fp16 x, each
    an f16 tensor or its bits in an int16 or uint16 one, on the matrix cores;
    asynchronous on stream."""
    dev = _device(w16, x16, y, offsets, x_rows, y_rows)
    i32 = _torch.int32
    x_count = rows if x_count is None else x_count
    y_count = rows if y_count is None else y_count
    halves = (_torch.float16, _torch.int16, _torch.uint16)
    for t in (w16, x16):
        if hasattr(t, "get_device") and t.dtype not in halves:
            raise TypeError("expected f16 (or its bits as 16-bit integers), got %s" % t.dtype)
    _run(load_library().q4k_f16_gemm_grouped, "q4k_f16_gemm_grouped", dev, stream,
         _at(w16, None, groups * n * k, dev), _at(x16, None, x_count * k, dev),
         _at(y, _torch.float32, y_count * n, dev), _at(offsets, i32, groups + 1, dev),
         _at(x_rows, i32, rows, dev), _at(y_rows, i32, rows, dev), int(n), int(k), int(groups),
         int(rows), int(x_div), int(x_count), int(y_count))


def q4k_lora_ws(rows: int, r: int) -> int:
    """Bytes of workspace of q4k_lora."""
    return int(load_library().q4k_lora_ws(int(rows), int(r)))


def q4k_lora(x, a, b, y, offsets, order, n: int, k: int, r: int, adapters: int, rows: int, *,
             base=None, ranks=None, scales=None, ws=None, ws_bytes=None, x_type=None,
             stream=None) -> None:
    """y[row] = base[row] + scales[a] B_a (A_a x[row]) for the rows of each
    adapter a (a: adapters x r x k, b: adapters x n x r, both f16; x f32, f16
    or bf16; offsets and order as q4k_moe_group gives them); asynchronous on
    stream."""
    dev = _device(x, a, b, y, offsets, order, base, ranks, scales, ws)
    f32, i32, f16 = _torch.float32, _torch.int32, _torch.float16
    _run(load_library().q4k_lora, "q4k_lora", dev, stream, _at(x, None, rows * k, dev),
         _act_type(x, x_type), _at(a, f16, adapters * r * k, dev),
         _at(b, f16, adapters * n * r, dev),
         _at(base, f32, rows * n, dev), _at(y, f32, rows * n, dev), _at(ranks, i32, adapters, dev),
         _at(scales, f32, adapters, dev), _at(offsets, i32, adapters + 1, dev),
         _at(order, i32, rows, dev), int(n), int(k), int(r), int(adapters), int(rows),
         _at(ws, None, 0, dev), _ws_bytes(ws, ws_bytes))


def q4k_read_calibrate_blocks() -> int:
    return int(load_library().q4k_read_calibrate_blocks())


def q4k_read_calibrate(buf, nbytes: int, out, stream=None) -> None:
    _check(load_library().q4k_read_calibrate(_addr(buf), int(nbytes), _addr(out), _stream(stream)),
           "q4k_read_calibrate")
