"""Python binding of libgemv (ctypes): argument marshalling only.

The names and argument order are those of ``include/gemv.h``:

    gemv_f32 (A, x, bias, y, M, K, B, stream=None)
    gemv_f16 (A, x, bias, y, M, K, B, stream=None)
    gemv_bf16(A, x, bias, y, M, K, B, stream=None)
    gemv_w8  (A, row_scale, x, bias, y, M, K, B, stream=None)
    gemv_f8  (A, a_scale, x, x_scale, bias, y, M, K, B, y_dtype="bf16", stream=None)
    gemv_f8_quantize(dtype, x, q, scale, K, B, stream=None)
    gemv_qk_norm_rope(dtype, q, k, q_out, k_out, q_weight, k_weight, inv_freq, lens, starts, S, N,
                      q_heads, k_heads, dim, rot, layout="half", eps=1e-6, factor=1.0, stream=None)
    gemv_kv8_append(dtype, *cache, k, v, lens, starts, S, N, stream=None)
    gemv_kv8_read  (dtype, *cache, k, v, lens, starts, S, N, stream=None)
    gemv_kv8_attention(dtype, *cache, q, lens, out, lse, S, T, q_heads, scale,
                       window=0, sinks=0, stream=None)
    gemv_kv8_prefix_attention(dtype, *cache, q, lens, firsts, prefix, out, lse, S, T, q_heads,
                              scale, stream=None)

(``cache``: k, v, k_scale, v_scale, table: tensors, whose shapes give the sizes; k, v and
q are tensors, too, whose strides give the distance of their rows).

Buffers may be torch CUDA tensors (checked for device, contiguity, element size
and minimum length before the call) or raw device addresses (ints, unchecked).
``bias`` may be None.  ``stream`` may be None (torch's current stream), a
``torch.cuda.Stream`` or a raw ``cudaStream_t`` value.  Every computation runs in
the CUDA library; a status other than GEMV_SUCCESS raises ``GemvError``.  There is
no fallback: without ``libgemv.so`` (build it with ``build()``) nothing runs.
"""
from __future__ import annotations

import ctypes
import os
import struct

from .build import LIB as LIB_PATH, build

__all__ = [
    "gemv_f32", "gemv_f16", "gemv_bf16", "gemv_w8", "gemv_w4", "gemv_bf16_splitk_noalloc", "gemv_ex",
    "gemv_swiglu", "gemv_host", "set_launch_overlap", "ACT_NONE", "ACT_SILU", "GemvError", "Plan", "plan_for",
    "status_string", "launch_count", "last_cuda_error", "force_kernel", "last_plan",
    "gemv_f8", "gemv_f8_quantize", "gemv_kv8_append", "gemv_kv8_read", "gemv_kv8_attention", "gemv_kv8_prefix_attention",
    "gemv_qk_norm_rope",
    "rope_frequencies", "F8_GROUP", "KV8_BLOCK",
    "KERNELS", "DTYPE_CODES", "lib", "build", "LIB_PATH", "device_status", "test_stall",
]

SUCCESS, ERR_INVALID_VALUE, ERR_UNSUPPORTED, ERR_CUDA, ERR_DEVICE_TIMEOUT = 0, 1, 2, 3, 4
MAX_BATCH, MAX_BATCH_TC = 16, 256
ACT_NONE, ACT_SILU = 0, 1
DTYPE_CODES = {"f32": 0, "f16": 1, "bf16": 2, "w8": 3, "w4": 4}
W4_GROUP = 128  # elements of a row that share one int4 scale
F8_GROUP = 128  # columns (and weight rows) that share one scale of an 8-bit floating point matrix
KV8_BLOCK = 64  # tokens of the 8-bit cache that share one scale (per head)
KERNELS = {"auto": 0, "rows_per_warp": 1, "warp_per_row": 2, "block_per_row": 3,
           "split_k": 4, "batched": 5, "scalar": 6, "stream": 7, "xsplit": 8, "tc": 9}
X_STAGING = {0: "global", 1: "smem", 2: "smem_fp32", 3: "regs"}
# BATCHED kernel variants (plan "variant"; force_kernel("batched", variant + 1))
BATCHED_ROWPAIR, BATCHED_RING, BATCHED_RING_MIXED = 0, 1, 2
KERNEL_NAMES = {v: k for k, v in KERNELS.items()}


class Plan(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int), ("lanes_per_row", ctypes.c_int),
                ("rows_per_warp", ctypes.c_int), ("splits", ctypes.c_int), ("unroll", ctypes.c_int),
                ("x_staging", ctypes.c_int), ("nb", ctypes.c_int),
                ("threads", ctypes.c_int), ("grid", ctypes.c_int64), ("smem_bytes", ctypes.c_int),
                ("workspace_bytes", ctypes.c_int64), ("variant", ctypes.c_int)]

    def as_dict(self) -> dict:
        d = {f: getattr(self, f) for f, _ in self._fields_}
        d["kernel_name"] = KERNEL_NAMES.get(self.kernel, "?")
        return d


# gemv_kv8_cache_t: k, v, k_scale, v_scale, table, blocks, width, heads, dim
KV8_CACHE = struct.Struct("@5P2q2i")


class GemvError(RuntimeError):
    def __init__(self, status: int, cuda_error: int = 0):
        self.status = status
        self.cuda_error = cuda_error
        msg = status_string(status)
        if status == ERR_CUDA:
            msg += f" (cudaError {cuda_error})"
        super().__init__(msg)


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libgemv.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: run decode_linear_layers_gb300.build()")
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, ci = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        for n in ("gemv_f32", "gemv_f16", "gemv_bf16"):
            f = getattr(L, n)
            f.argtypes = [vp, vp, vp, vp, i64, i64, ci, vp]
            f.restype = ci
        L.gemv_w8.argtypes = [vp, vp, vp, vp, vp, i64, i64, ci, vp]
        L.gemv_w8.restype = ci
        L.gemv_w4.argtypes = [vp, vp, vp, vp, vp, i64, i64, ci, vp]
        L.gemv_w4.restype = ci
        L.gemv_bf16_splitk_noalloc.argtypes = [vp, vp, vp, vp, i64, i64, ci, vp]
        L.gemv_bf16_splitk_noalloc.restype = ci
        L.gemv_ex.argtypes = [ci, vp, vp, vp, vp, vp, vp, i64, i64, ci, ci, vp]
        L.gemv_ex.restype = ci
        L.gemv_swiglu.argtypes = [ci, vp, vp, vp, vp, vp, i64, i64, ci, vp]
        L.gemv_swiglu.restype = ci
        L.gemv_host.argtypes = [ci, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, ci, vp]
        L.gemv_host.restype = ci
        L.gemv_f8_quantize.argtypes = [ci, vp, vp, vp, i64, ci, vp]
        L.gemv_f8_quantize.restype = ci
        L.gemv_f8.argtypes = [vp, vp, vp, vp, vp, vp, ci, i64, i64, ci, vp]
        L.gemv_f8.restype = ci
        L.gemv_kv8_append.argtypes = [ci, vp, vp, i64, vp, i64, vp, vp, ci, i64, vp]
        L.gemv_kv8_append.restype = ci
        L.gemv_kv8_read.argtypes = [ci, vp, vp, i64, vp, i64, vp, vp, ci, i64, vp]
        L.gemv_kv8_read.restype = ci
        cf, cd = ctypes.c_float, ctypes.c_double
        L.gemv_qk_norm_rope.argtypes = ([ci] + [vp, i64, vp, i64, vp, ci] * 2 + [ci, cf, vp, ci, ci, cf, vp, vp, ci, i64, vp])
        L.gemv_qk_norm_rope.restype = ci
        L.gemv_rope_frequencies.argtypes = [ctypes.POINTER(cf), ci, cd, ci, cd, cd, cd, cd, ctypes.POINTER(cf)]
        L.gemv_rope_frequencies.restype = ci
        L.gemv_kv8_attention.argtypes = [ci, vp, vp, i64, vp, vp, vp, ci, ci, ci, ctypes.c_float, i64, i64, vp]
        L.gemv_kv8_attention.restype = ci
        L.gemv_kv8_prefix_attention.argtypes = [ci, vp, vp, i64, vp, vp, vp, ci, vp, vp, ci, ci, ci, cf, vp]
        L.gemv_kv8_prefix_attention.restype = ci
        L.gemv_set_launch_overlap.argtypes = [ci]
        L.gemv_set_launch_overlap.restype = ci
        L.gemv_status_string.argtypes = [ci]
        L.gemv_status_string.restype = ctypes.c_char_p
        L.gemv_last_cuda_error.argtypes = []
        L.gemv_last_cuda_error.restype = ci
        L.gemv_launch_count.argtypes = []
        L.gemv_launch_count.restype = ctypes.c_uint64
        L.gemv_plan_for.argtypes = [ci, i64, i64, ci, ci, ci, ctypes.POINTER(Plan)]
        L.gemv_plan_for.restype = ci
        L.gemv_test_force_kernel.argtypes = [ci, ci]
        L.gemv_test_force_kernel.restype = ci
        L.gemv_test_last_plan.argtypes = [ctypes.POINTER(Plan)]
        L.gemv_test_last_plan.restype = ci
        L.gemv_get_device_status.argtypes = [vp, ctypes.POINTER(ci)]
        L.gemv_get_device_status.restype = ci
        L.gemv_test_stall.argtypes = [ci, i64]
        L.gemv_test_stall.restype = ci
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().gemv_status_string(int(status)).decode()


def last_cuda_error() -> int:
    return int(lib().gemv_last_cuda_error())


def launch_count() -> int:
    return int(lib().gemv_launch_count())


def plan_for(dtype: str, M: int, K: int, B: int, aligned16: bool = True, num_sms: int = 152) -> dict:
    p = Plan()
    st = lib().gemv_plan_for(DTYPE_CODES[dtype], int(M), int(K), int(B), int(bool(aligned16)),
                             int(num_sms), ctypes.byref(p))
    if st != SUCCESS:
        raise GemvError(st)
    return p.as_dict()


def device_status(stream=None) -> tuple:
    """Synchronise `stream` and read (then clear) the device status word of the
    kernels with bounded waits and of the 8-bit cache: (status, bits), status SUCCESS,
    ERR_DEVICE_TIMEOUT or ERR_INVALID_VALUE (a block that the cache's pool or table does
    not have); raises GemvError on a CUDA failure."""
    bits = ctypes.c_int(0)
    st = lib().gemv_get_device_status(_stream(stream), ctypes.byref(bits))
    if st not in (SUCCESS, ERR_DEVICE_TIMEOUT, ERR_INVALID_VALUE):
        _check(st)
    return st, int(bits.value)


def test_stall(stall: int, timeout_ns: int = 0) -> None:
    """TEST ONLY: make later tensor-core launches skip their first CTA's last MMA,
    so that CTA's wait runs out after timeout_ns (<= 0: 2 s).  2, 3: where gemv_f8 runs on
    pairs of SMs, the last copies of the first pair's first or second CTA instead."""
    _check(lib().gemv_test_stall(int(stall), int(timeout_ns)))


def force_kernel(kernel, param: int = 0) -> None:
    """TEST ONLY: force a kernel family ("auto" restores dispatch)."""
    k = KERNELS[kernel] if isinstance(kernel, str) else int(kernel)
    st = lib().gemv_test_force_kernel(k, int(param))
    if st != SUCCESS:
        raise GemvError(st)


def last_plan() -> dict:
    """TEST ONLY: the plan of this thread's last successful call."""
    p = Plan()
    st = lib().gemv_test_last_plan(ctypes.byref(p))
    if st != SUCCESS:
        raise GemvError(st)
    return p.as_dict()


# ------------------------------------------------------------------ marshalling
def _addr(t, elem_size: int, min_elems: int, what: str):
    """Device address of a tensor (checked) or of a raw int pointer (unchecked)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    try:  # a tensor as it should be; what is wrong with another is said below
        if t.is_cuda and t.element_size() == elem_size and t.numel() >= min_elems and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    if not getattr(t, "is_cuda", False):
        raise ValueError(f"{what} must be a CUDA tensor or a device address")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if t.element_size() != elem_size:
        raise ValueError(f"{what}: element size {t.element_size()} != {elem_size}")
    if t.numel() < min_elems:
        raise ValueError(f"{what}: {t.numel()} elements < {min_elems} needed")
    return t.data_ptr()


_current_raw_stream = None  # (torch's current stream of the current device, as a handle)


def _stream(stream):
    global _current_raw_stream
    if stream is None:
        # the raw handle straight from torch (a Stream object per call costs microseconds)
        if _current_raw_stream is None:
            import torch
            get = getattr(torch._C, "_cuda_getCurrentRawStream", None)
            dev = torch._C._cuda_getDevice
            _current_raw_stream = ((lambda: get(dev())) if get is not None
                                   else (lambda: torch.cuda.current_stream().cuda_stream))
        return _current_raw_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(st: int) -> None:
    if st != SUCCESS:
        raise GemvError(st, last_cuda_error() if st == ERR_CUDA else 0)


def _sizes(M, K, B):
    M, K, B = int(M), int(K), int(B)
    if min(M, K, B) < 0:
        return M, K, B, 0, 0, 0  # let the library report the bad size
    return M, K, B, M * K, B * K, B * M


_entry = {}  # entry points by name, looked up once


def _fn(name):
    f = _entry.get(name)
    if f is None:
        f = _entry[name] = getattr(lib(), name)
    return f


def _float_gemv(name, esize, A, x, bias, y, M, K, B, stream):
    M, K, B, na, nx, ny = _sizes(M, K, B)
    args = (_addr(A, esize, na, "A"), _addr(x, esize, nx, "x"),
            _addr(bias, esize, M if bias is not None else 0, "bias"),
            _addr(y, esize, ny, "y"))
    _check(_fn(name)(*args, M, K, B, _stream(stream)))


def gemv_f32(A, x, bias, y, M, K, B, stream=None) -> None:
    """y[b, m] = sum_k A[m, k] x[b, k] (+ bias[m]); fp32 storage and accumulation."""
    _float_gemv("gemv_f32", 4, A, x, bias, y, M, K, B, stream)


def gemv_f16(A, x, bias, y, M, K, B, stream=None) -> None:
    """fp16 storage (torch.float16), fp32 accumulation, fp16 output."""
    _float_gemv("gemv_f16", 2, A, x, bias, y, M, K, B, stream)


def gemv_bf16(A, x, bias, y, M, K, B, stream=None) -> None:
    """bf16 storage (torch.bfloat16), fp32 accumulation, bf16 output."""
    _float_gemv("gemv_bf16", 2, A, x, bias, y, M, K, B, stream)


def gemv_w8(A, row_scale, x, bias, y, M, K, B, stream=None) -> None:
    """int8 A with fp32 row_scale; bf16 x, bias and y; fp32 accumulation."""
    M, K, B, na, nx, ny = _sizes(M, K, B)
    args = (_addr(A, 1, na, "A"), _addr(row_scale, 4, M, "row_scale"), _addr(x, 2, nx, "x"),
            _addr(bias, 2, M if bias is not None else 0, "bias"), _addr(y, 2, ny, "y"))
    _check(_fn("gemv_w8")(*args, M, K, B, _stream(stream)))


OVERLAP = {"off": 0, "launch": 1, "weights": 2}


def set_launch_overlap(mode: str) -> None:
    """Launch overlap for this thread's later calls: "off", "launch" (programmatic
    dependent launches, every access after the previous kernel; the default) or
    "weights" (the first weight loads before that wait; only for weights the
    preceding work does not write)."""
    _check(lib().gemv_set_launch_overlap(OVERLAP[mode]))


def _host_addr(t, elem_size: int, min_elems: int, what: str):
    """Host address of a CPU tensor (checked) or of a raw int pointer (unchecked)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if getattr(t, "is_cuda", True):
        raise ValueError(f"{what} must be a CPU tensor (pinned for asynchronous copies) or a host address")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if t.element_size() != elem_size:
        raise ValueError(f"{what}: element size {t.element_size()} != {elem_size}")
    if t.numel() < min_elems:
        raise ValueError(f"{what}: {t.numel()} elements < {min_elems} needed")
    return t.data_ptr()


def gemv_host(dtype, h_A, h_scale, h_x, h_bias, h_y, d_A, d_scale, d_x, d_bias, d_y, M, K, B,
              stream=None) -> None:
    """The GEMV on host buffers: copies h_A, h_scale, h_x, h_bias (CPU tensors,
    pinned for asynchronous copies; None skips a copy) into the device buffers d_*,
    runs it there and copies y back into h_y, all enqueued on `stream`."""
    M, K, B, _, nx, ny = _sizes(M, K, B)
    sa = {"f32": 4, "f16": 2, "bf16": 2, "w8": 1, "w4": 1}[dtype]
    sx = 4 if dtype == "f32" else 2
    na, ns = _a_count(dtype, M, K)
    hs = (_host_addr(h_A, sa, na, "h_A"), _host_addr(h_scale, 4, ns, "h_scale"), _host_addr(h_x, sx, nx, "h_x"),
          _host_addr(h_bias, sx, M if h_bias is not None else 0, "h_bias"), _host_addr(h_y, sx, ny, "h_y"))
    ds = (_addr(d_A, sa, na, "d_A"), _addr(d_scale, 4, ns, "d_scale"), _addr(d_x, sx, nx, "d_x"),
          _addr(d_bias, sx, M if d_bias is not None else 0, "d_bias"), _addr(d_y, sx, ny, "d_y"))
    _check(lib().gemv_host(DTYPE_CODES[dtype], *hs, *ds, M, K, B, _stream(stream)))


NOALLOC_SCRATCH_BYTES = 4 * 1024 * 1024


def gemv_w4(A, group_scale, x, bias, y, M, K, B, stream=None) -> None:
    """int4 A, two per byte (torch.uint8, M x K/2, even element in the low nibble),
    with fp32 group_scale (M x K/W4_GROUP); bf16 x, bias and y; fp32 accumulation."""
    M, K, B, _, nx, ny = _sizes(M, K, B)
    na, ns = _a_count("w4", M, K)
    args = (_addr(A, 1, na, "A"), _addr(group_scale, 4, ns, "group_scale"), _addr(x, 2, nx, "x"),
            _addr(bias, 2, M if bias is not None else 0, "bias"), _addr(y, 2, ny, "y"))
    _check(_fn("gemv_w4")(*args, M, K, B, _stream(stream)))


def gemv_bf16_splitk_noalloc(A, x, bias, y, M, K, B, stream=None) -> None:
    """gemv_bf16 on the split-K path with its partial sums in the library's fixed
    device array (no device allocation).  For callers that cannot allocate while
    they run; calls that overlap on the GPU race on the shared array.  Raises
    GemvError(GEMV_ERR_UNSUPPORTED) when splits x B x M x 4 bytes exceed
    NOALLOC_SCRATCH_BYTES or the rows are not 16-byte aligned."""
    _float_gemv("gemv_bf16_splitk_noalloc", 2, A, x, bias, y, M, K, B, stream)


_ESIZE = {"f32": (4, 4), "f16": (2, 2), "bf16": (2, 2), "w8": (1, 2), "w4": (1, 2)}   # (A, x/bias/y)


def _a_count(dtype, M, K):
    """Elements of A's storage (bytes for int4, two values each) and of its scales."""
    if dtype == "w4":
        return max(0, M * K // 2), max(0, M * (K // W4_GROUP))
    return max(0, M * K), max(0, M)


def gemv_ex(dtype, A, row_scale, x, bias, residual, y, M, K, B, act=ACT_NONE, stream=None) -> None:
    """y = act(s_m * sum_k A x + bias) + residual, one launch, any storage type.

    row_scale: w8 only (else None).  residual: (B, M) in y's type, None, or y itself
    (in place)."""
    M, K, B, _, nx, ny = _sizes(M, K, B)
    na, ns = _a_count(dtype, M, K)
    sa, sx = _ESIZE[dtype]
    args = (_addr(A, sa, na, "A"), _addr(row_scale, 4, ns, "row_scale"), _addr(x, sx, nx, "x"),
            _addr(bias, sx, M if bias is not None else 0, "bias"),
            _addr(residual, sx, ny if residual is not None else 0, "residual"), _addr(y, sx, ny, "y"))
    _check(_fn("gemv_ex")(DTYPE_CODES[dtype], *args, M, K, B, int(act), _stream(stream)))


def gemv_swiglu(dtype, A, row_scale, x, bias, y, I, K, B, stream=None) -> None:
    """y[b][m] = silu(gate_m) * up_m over A = [gate rows; up rows] (2I x K)."""
    I, K, B = int(I), int(K), int(B)
    M2 = 2 * I if I >= 0 else 0
    sa, sx = _ESIZE[dtype]
    na, ns = _a_count(dtype, M2, K)
    args = (_addr(A, sa, na, "A"), _addr(row_scale, 4, ns, "row_scale"),
            _addr(x, sx, max(0, B * K), "x"), _addr(bias, sx, M2 if bias is not None else 0, "bias"),
            _addr(y, sx, max(0, B * I), "y"))
    _check(_fn("gemv_swiglu")(DTYPE_CODES[dtype], *args, I, K, B, _stream(stream)))


# ------------------------------------------------------ 8-bit floating point layers
def gemv_f8_quantize(dtype, x, q, scale, K, B, stream=None) -> None:
    """x (B, K) of `dtype` ("f32", "f16", "bf16") to e4m3 values q and fp32 scales
    (B, ceil(K / F8_GROUP)), one for each group of F8_GROUP elements of a vector."""
    K, B = int(K), int(B)
    n, g = max(0, B * K), max(0, B * -(-K // F8_GROUP))
    args = (_addr(x, _ESIZE[dtype][1], n, "x"), _addr(q, 1, n, "q"), _addr(scale, 4, g, "scale"))
    _check(_fn("gemv_f8_quantize")(DTYPE_CODES[dtype], *args, K, B, _stream(stream)))


def gemv_f8(A, a_scale, x, x_scale, bias, y, M, K, B, y_dtype="bf16", stream=None) -> None:
    """y[b, m] = sum_k (a_scale A)[m, k] (x_scale x)[b, k] (+ bias[m]): e4m3 A (M, K)
    with a scale for each block of F8_GROUP x F8_GROUP, e4m3 x (B, K) with one for each
    F8_GROUP elements of a vector; y and bias of `y_dtype`."""
    M, K, B, na, nx, ny = _sizes(M, K, B)
    G, sy = -(-max(K, 0) // F8_GROUP), _ESIZE[y_dtype][1]
    args = (_addr(A, 1, na, "A"), _addr(a_scale, 4, -(-max(M, 0) // F8_GROUP) * G, "a_scale"), _addr(x, 1, nx, "x"),
            _addr(x_scale, 4, max(0, B * G), "x_scale"), _addr(bias, sy, M if bias is not None else 0, "bias"),
            _addr(y, sy, ny, "y"))
    _check(_fn("gemv_f8")(*args, DTYPE_CODES[y_dtype], M, K, B, _stream(stream)))


ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "base": 2, "turns": 3, "index": 4}


def rope_frequencies(rot, base=10000.0, scaling="none", factor=1.0, original=0.0, low=1.0, high=32.0) -> tuple:
    """(rot / 2 floats for gemv_qk_norm_rope's inv_freq, its `factor`), worked out on the
    host: base^(-2 i / rot), for a context `factor` times as long as `original` tokens by
    "linear", "base", "turns" (low, high: turns of a pair in the original context) or
    "index" scaling."""
    freq, att = (ctypes.c_float * max(1, rot // 2))(), ctypes.c_float(1.0)
    _check(lib().gemv_rope_frequencies(freq, int(rot), float(base), ROPE_SCALINGS[scaling], float(factor), float(original),
                                       float(low), float(high), ctypes.byref(att)))
    return list(freq)[:rot // 2], float(att.value)


def gemv_qk_norm_rope(dtype, q, k, q_out, k_out, q_weight, k_weight, inv_freq, lens, starts, S, N, q_heads, k_heads, dim,
                      rot, layout="half", eps=1e-6, factor=1.0, stream=None) -> None:
    """Norm (over each head's dim channels, with q_weight and k_weight; None: none) and
    rotation by the position of N rows of queries (q_heads x dim of `dtype`) and keys
    (k_heads x dim): pair i of the first `rot` channels, (i, i + rot / 2) ("half") or
    (2 i, 2 i + 1) ("interleaved"), by position x inv_freq[i] (fp32), cos and sin times
    `factor`.  lens and starts (int32) say where the rows stand, as gemv_kv8_append takes
    them.  q, k, q_out and k_out may be columns of wider tensors; an output of None means in
    place; k may be None with k_heads == 0, and q with q_heads == 0."""
    S, N, q_heads, k_heads, dim, rot = int(S), int(N), int(q_heads), int(k_heads), int(dim), int(rot)
    size, n = _ESIZE[dtype][1], max(N, 0)
    sides = []
    for x, y, w, heads, what in ((q, q_out, q_weight, q_heads, "q"), (k, k_out, k_weight, k_heads, "k")):
        row = max(0, heads * dim)
        if row == 0 and x is None:
            sides += [None, 0, None, 0, None, heads]
            continue
        xa, xs = _rows(x, size, n, row, what)
        ya, ys = (xa, xs) if y is None else _rows(y, size, n, row, what + "_out")
        sides += [xa, xs, ya, ys, _addr(w, size, max(dim, 0), what + "_weight"), heads]
    _check(_fn("gemv_qk_norm_rope")(DTYPE_CODES[dtype], *sides, dim, float(eps), _addr(inv_freq, 4, max(0, rot // 2), "inv_freq"),
                                    rot, ROPE_LAYOUTS[layout], float(factor), _addr(lens, 4, max(S, 0), "lens"),
                                    _addr(starts, 4, S + 1, "starts"), S, N, _stream(stream)))


def _kv8_cache(k, v, k_scale, v_scale, table, S):
    """The cache as the library takes it (packed), heads and dim; sizes from the
    tensors' shapes."""
    ks, vs, ts = k.shape, v.shape, table.shape
    if len(ks) != 4 or ks[2] != KV8_BLOCK or vs != (ks[0], ks[1], ks[3], KV8_BLOCK):
        raise ValueError(f"k must be (blocks, heads, {KV8_BLOCK}, dim) and v (blocks, heads, dim, {KV8_BLOCK}): "
                         f"got {tuple(ks)} and {tuple(vs)}")
    if len(ts) != 2 or ts[0] < S:
        raise ValueError(f"table must be ({S}, width): got {tuple(ts)}")
    blocks, heads, _, dim = ks
    n = blocks * heads
    return KV8_CACHE.pack(_addr(k, 1, 0, "k"), _addr(v, 1, 0, "v"), _addr(k_scale, 4, n, "k_scale"),
                          _addr(v_scale, 4, n, "v_scale"), _addr(table, 4, 0, "table"), blocks, ts[1], heads, dim), heads, dim


def _rows(t, elem_size, rows, row, what):
    """Address and row stride of a tensor whose last dimensions, flattened, are rows of
    `row` consecutive elements and whose first ones are `rows` evenly spaced rows."""
    if not getattr(t, "is_cuda", False):
        raise ValueError(f"{what} must be a CUDA tensor")
    if t.element_size() != elem_size:
        raise ValueError(f"{what}: element size {t.element_size()} != {elem_size}")
    if t.numel() != rows * row:
        raise ValueError(f"{what}: {t.numel()} elements, {rows} rows of {row} are needed")
    if t.is_contiguous() or rows == 0:
        return t.data_ptr(), row
    st = t.stride()
    if len(st) == 3 and st[2] == 1 and t.shape[0] == rows > 1 and st[1] == t.shape[2]:  # rows of heads x dim
        return t.data_ptr(), st[0]
    if rows == 1:  # one row: its own dimensions alone have to be consecutive
        stride = row
    else:
        stride = None
    want, n = 1, 1  # expected stride, elements covered so far
    for size, st in zip(reversed(t.shape), reversed(t.stride())):
        if size == 1:
            continue
        if n == row:  # the innermost of the row dimensions
            if stride is None:
                stride = want = st
        if st != want:
            raise ValueError(f"{what}: strides {t.stride()} are no evenly spaced rows of {row} consecutive elements")
        want *= size
        n *= size
    return t.data_ptr(), stride


def gemv_kv8_append(dtype, k_cache, v_cache, k_scale, v_scale, table, k, v, lens, starts, S, N, stream=None) -> None:
    """Writes N new tokens (rows of k and v, each heads x dim of `dtype`, columns of a
    wider tensor as well) to the 8-bit cache: those of sequence s are the rows
    starts[s] .. starts[s + 1] (int32, S + 1 values; None: N / S each) and take the last
    positions of its lens[s] tokens (int32)."""
    S, N = int(S), int(N)
    cache, heads, dim = _kv8_cache(k_cache, v_cache, k_scale, v_scale, table, S)
    size, row = _ESIZE[dtype][1], heads * dim
    ka, ks = _rows(k, size, max(N, 0), row, "k")
    va, vs = _rows(v, size, max(N, 0), row, "v")
    _check(_fn("gemv_kv8_append")(DTYPE_CODES[dtype], cache, ka, ks, va, vs, _addr(lens, 4, max(S, 0), "lens"),
                                  _addr(starts, 4, S + 1, "starts"), S, N, _stream(stream)))


def gemv_kv8_read(dtype, k_cache, v_cache, k_scale, v_scale, table, k, v, lens, starts, S, N, stream=None) -> None:
    """Cached tokens as N rows of k and v (each heads x dim of `dtype`, columns of a wider
    tensor as well; None: not read): the rows starts[s] .. starts[s + 1] (int32, S + 1
    values; None: N / S each) are the last ones of the lens[s] tokens of sequence s."""
    S, N = int(S), int(N)
    cache, heads, dim = _kv8_cache(k_cache, v_cache, k_scale, v_scale, table, S)
    size, row = _ESIZE[dtype][1], heads * dim
    ka, ks = (None, 0) if k is None else _rows(k, size, max(N, 0), row, "k")
    va, vs = (None, 0) if v is None else _rows(v, size, max(N, 0), row, "v")
    _check(_fn("gemv_kv8_read")(DTYPE_CODES[dtype], cache, ka, ks, va, vs, _addr(lens, 4, max(S, 0), "lens"),
                                _addr(starts, 4, S + 1, "starts"), S, N, _stream(stream)))


def gemv_kv8_attention(dtype, k_cache, v_cache, k_scale, v_scale, table, q, lens, out, lse, S, T, q_heads, scale,
                       window=0, sinks=0, stream=None) -> None:
    """Attention of the newest T tokens of S sequences over the 8-bit cache: q and out
    (S, T, q_heads, dim) of `dtype` ("f16", "bf16"; q also as columns of a wider
    tensor), lens (S) int32, lse (S, T, q_heads) fp32 or None.  window > 0: a query sees
    the `window` latest tokens, itself among them, and the first `sinks`."""
    S, T, q_heads = int(S), int(T), int(q_heads)
    cache, _, dim = _kv8_cache(k_cache, v_cache, k_scale, v_scale, table, S)
    size, rows, row = _ESIZE[dtype][1], max(0, S * T), max(0, q_heads * dim)
    qa, qs = _rows(q, size, rows, row, "q")
    _check(_fn("gemv_kv8_attention")(DTYPE_CODES[dtype], cache, qa, qs, _addr(lens, 4, max(S, 0), "lens"),
                                     _addr(out, size, rows * row, "out"),
                                     _addr(lse, 4, rows * max(q_heads, 0), "lse"), S, T, q_heads, float(scale),
                                     int(window), int(sinks), _stream(stream)))


def gemv_kv8_prefix_attention(dtype, k_cache, v_cache, k_scale, v_scale, table, q, lens, firsts, prefix, out, lse, S, T,
                              q_heads, scale, stream=None) -> None:
    """gemv_kv8_attention (no window) for groups of sequences whose tables begin with the
    same blocks, read once for all of a group's queries: group g has the sequences
    firsts[g] .. firsts[g + 1] (int32, groups + 1 values; None: one group of all), which have
    their first prefix[g] tokens (int32; one value for each group) in common.  lens counts
    all tokens of a sequence, the prefix among them."""
    S, T, q_heads = int(S), int(T), int(q_heads)
    cache, _, dim = _kv8_cache(k_cache, v_cache, k_scale, v_scale, table, S)
    size, rows, row = _ESIZE[dtype][1], max(0, S * T), max(0, q_heads * dim)
    if isinstance(prefix, int):
        raise ValueError("prefix must be a tensor: it has a value for each group")
    groups = prefix.numel()
    qa, qs = _rows(q, size, rows, row, "q")
    _check(_fn("gemv_kv8_prefix_attention")(DTYPE_CODES[dtype], cache, qa, qs, _addr(lens, 4, max(S, 0), "lens"),
                                            _addr(firsts, 4, groups + 1, "firsts"), _addr(prefix, 4, groups, "prefix"), groups,
                                            _addr(out, size, rows * row, "out"),
                                            _addr(lse, 4, rows * max(q_heads, 0), "lse"), S, T, q_heads, float(scale),
                                            _stream(stream)))
