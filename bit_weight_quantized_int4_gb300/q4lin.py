"""Thin ctypes binding of libq4lin.so, with the C ABI's names (include/q4lin.h).

Argument marshalling only: every step of the computation runs in the library's CUDA
kernels.  If the library has not been built this module raises at import time; there
is no fallback of any kind.

``q4lin_run`` and friends take raw integers for pointers and the stream.  ``linear``
is a convenience that takes torch CUDA tensors, checks their dtypes/shapes/contiguity,
and passes their data pointers and the current stream to ``q4lin_run``.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import NamedTuple, Optional

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libq4lin.so")
if not os.path.exists(_LIB_PATH):
    raise ImportError(
        f"{_LIB_PATH} is missing: build it with `python -m bit_weight_quantized_int4_gb300.build` "
        "(the q4lin CUDA library is required; there is no fallback)")
_lib = ctypes.CDLL(_LIB_PATH)

# ---- constants (mirror include/q4lin.h) ----
Q4LIN_OK = 0
Q4LIN_ERR_INVALID_ARG = 1
Q4LIN_ERR_UNSUPPORTED = 2
Q4LIN_ERR_CUDA = 3
Q4LIN_ERR_TIMEOUT = 4
Q4LIN_ERR_NO_DEVICE = 5
Q4LIN_ERR_TOO_LARGE = 6

Q4LIN_SCALE_F32 = 0
Q4LIN_SCALE_F16 = 1

Q4LIN_PATH_AUTO = 0
Q4LIN_PATH_GEMV = 1
Q4LIN_PATH_FFMA = 2
Q4LIN_PATH_TC = 3
Q4LIN_PATH_TC_SMALL = 4
PATH_NAMES = {0: "auto", 1: "gemv", 2: "ffma", 3: "tc", 4: "tc_small"}

Q4LIN_KERNEL_NONE = 0
Q4LIN_KERNEL_GEMV_TMA = 1
Q4LIN_KERNEL_MULTIROW = 2
Q4LIN_KERNEL_ROWSTREAM = 3
Q4LIN_KERNEL_GENERIC = 4
Q4LIN_KERNEL_TC = 5
Q4LIN_KERNEL_TC_F16 = 6
Q4LIN_KERNEL_GEMV_TMA_FIXED = 7
Q4LIN_KERNEL_TC_SMALL = 8
Q4LIN_KERNEL_TC_SMALL_BF16 = 9
KERNEL_NAMES = {0: "none", 1: "gemv_tma", 2: "multirow", 3: "rowstream", 4: "generic",
                5: "tc", 6: "tc_f16", 7: "gemv_tma_fixed", 8: "tc_small", 9: "tc_small_bf16"}

Q4LIN_DTYPE_F32 = 0
Q4LIN_DTYPE_F16 = 1
Q4LIN_DTYPE_BF16 = 2

Q4LIN_OPT_FORCE_PATH = 1
Q4LIN_OPT_NIBBLE_EVEN_HIGH = 2
Q4LIN_OPT_WAIT_LIMIT = 3
Q4LIN_OPT_PDL = 4
Q4LIN_OPT_TC_SKIP_FIRST_COPY = 5
Q4LIN_OPT_TC_F16 = 6
Q4LIN_OPT_TC_SMALL_OPERANDS = 7
Q4LIN_OPT_ATTENTION_SPLIT_ROWS = 8

_vp, _i64, _i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int

_lib.q4lin_create.argtypes = [ctypes.POINTER(_vp), _i32]
_lib.q4lin_create.restype = _i32
_lib.q4lin_destroy.argtypes = [_vp]
_lib.q4lin_destroy.restype = _i32
_lib.q4lin_run.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i32, _vp]
_lib.q4lin_run.restype = _i32
class q4lin_problem_t(ctypes.Structure):
    _fields_ = [("x", _vp), ("qweight", _vp), ("scales", _vp), ("bias", _vp), ("out", _vp),
                ("M", _i64), ("N", _i64), ("K", _i64), ("group_size", _i64),
                ("scale_dtype", _i32)]


_lib.q4lin_run_grouped.argtypes = [_vp, ctypes.POINTER(q4lin_problem_t), _i32, _vp]
_lib.q4lin_run_grouped.restype = _i32
_lib.q4lin_run_static_scratch.argtypes = [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i32, _vp]
_lib.q4lin_run_static_scratch.restype = _i32
_lib.q4lin_run_backward_dx.argtypes = [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i32,
                                       _vp]
_lib.q4lin_run_backward_dx.restype = _i32
_lib.q4lin_run_requant.argtypes = [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _i32, _vp]
_lib.q4lin_run_requant.restype = _i32


class q4lin_kv_cache_t(ctypes.Structure):
    _fields_ = [("k_codes", _vp), ("k_scales", _vp), ("v_codes", _vp), ("v_scales", _vp),
                ("page_table", _vp), ("num_pages", _i64), ("kv_heads", _i64),
                ("page_size", _i64), ("head_dim", _i64), ("batch", _i64),
                ("pages_per_sequence", _i64), ("table_stride", _i64)]


class q4lin_rope_t(ctypes.Structure):
    _fields_ = [("cos", _vp), ("sin", _vp), ("positions", _i64), ("rotated", _i64),
                ("interleaved", _i32)]


class q4lin_kv_append_t(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("k_token_stride", _i64), ("k_head_stride", _i64),
                ("v_token_stride", _i64), ("v_head_stride", _i64), ("dtype", _i32),
                ("tokens", _i64), ("offsets", _vp), ("starts", _vp), ("rope", q4lin_rope_t)]


class q4lin_attention_t(ctypes.Structure):
    _fields_ = [("query", _vp), ("q_token_stride", _i64), ("q_head_stride", _i64), ("out", _vp),
                ("lse", _vp), ("dtype", _i32), ("tokens", _i64), ("heads", _i64),
                ("max_query", _i64), ("offsets", _vp), ("lengths", _vp),
                ("scale", ctypes.c_float), ("causal", _i32), ("window", _i64),
                ("rope", q4lin_rope_t)]


class q4lin_kv_read_t(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("dtype", _i32), ("tokens", _i64), ("offsets", _vp),
                ("starts", _vp)]


class q4lin_norm_rope_t(ctypes.Structure):
    _fields_ = [("q", _vp), ("k", _vp), ("q_token_stride", _i64), ("q_head_stride", _i64),
                ("k_token_stride", _i64), ("k_head_stride", _i64), ("q_weight", _vp),
                ("k_weight", _vp), ("q_out", _vp), ("k_out", _vp), ("q_out_token_stride", _i64),
                ("q_out_head_stride", _i64), ("k_out_token_stride", _i64),
                ("k_out_head_stride", _i64), ("dtype", _i32), ("tokens", _i64), ("heads", _i64),
                ("kv_heads", _i64), ("head_dim", _i64), ("positions", _vp),
                ("rope", q4lin_rope_t), ("eps", ctypes.c_float)]


class q4lin_norm_rope_backward_t(ctypes.Structure):
    _fields_ = [("forward", q4lin_norm_rope_t), ("d_q_out", _vp), ("d_k_out", _vp),
                ("d_q_out_token_stride", _i64), ("d_q_out_head_stride", _i64),
                ("d_k_out_token_stride", _i64), ("d_k_out_head_stride", _i64),
                ("d_q_weight", _vp), ("d_k_weight", _vp)]


class q4lin_logprobs_t(ctypes.Structure):
    _fields_ = [("logits", _vp), ("row_stride", _i64), ("dtype", _i32), ("rows", _i64),
                ("vocabulary", _i64), ("tokens", _vp), ("logprob", _vp), ("entropy", _vp),
                ("lse", _vp), ("top", _i64), ("top_tokens", _vp), ("top_logprobs", _vp)]


class q4lin_logprobs_backward_t(ctypes.Structure):
    _fields_ = [("logits", _vp), ("row_stride", _i64), ("dtype", _i32), ("rows", _i64),
                ("vocabulary", _i64), ("tokens", _vp), ("lse", _vp), ("entropy", _vp),
                ("d_logprob", _vp), ("d_entropy", _vp), ("d_logits", _vp),
                ("d_row_stride", _i64)]


for _name, _types in (("q4lin_run_kv_append", (q4lin_kv_cache_t, q4lin_kv_append_t)),
                      ("q4lin_run_attention", (q4lin_kv_cache_t, q4lin_attention_t)),
                      ("q4lin_run_kv4_append", (q4lin_kv_cache_t, q4lin_kv_append_t)),
                      ("q4lin_run_kv4_read", (q4lin_kv_cache_t, q4lin_kv_read_t)),
                      ("q4lin_run_kv4_attention", (q4lin_kv_cache_t, q4lin_attention_t)),
                      ("q4lin_run_norm_rope", (q4lin_norm_rope_t,)),
                      ("q4lin_run_norm_rope_backward", (q4lin_norm_rope_backward_t,)),
                      ("q4lin_run_logprobs", (q4lin_logprobs_t,)),
                      ("q4lin_run_logprobs_backward", (q4lin_logprobs_backward_t,))):
    _f = getattr(_lib, _name)
    _f.argtypes = [_vp, *(ctypes.POINTER(t) for t in _types), _vp]
    _f.restype = _i32
_lib.q4lin_plan.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i32,
                            ctypes.POINTER(_i32)]
_lib.q4lin_plan.restype = _i32
_lib.q4lin_plan_kernel.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i32,
                                   ctypes.POINTER(_i32)]
_lib.q4lin_plan_kernel.restype = _i32
_lib.q4lin_set_option.argtypes = [_vp, _i32, _i64]
_lib.q4lin_set_option.restype = _i32
_lib.q4lin_get_option.argtypes = [_vp, _i32, ctypes.POINTER(_i64)]
_lib.q4lin_get_option.restype = _i32
_lib.q4lin_check_device_status.argtypes = [_vp, _vp, ctypes.POINTER(_i32)]
_lib.q4lin_check_device_status.restype = _i32
_lib.q4lin_status_string.argtypes = [_i32]
_lib.q4lin_status_string.restype = ctypes.c_char_p


class Q4LinError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {q4lin_status_string(status)} (status {status})")
        self.status = status


def library_path() -> str:
    return _LIB_PATH


def q4lin_status_string(status: int) -> str:
    return _lib.q4lin_status_string(int(status)).decode()


def q4lin_create(device: int = 0) -> int:
    h = _vp()
    st = _lib.q4lin_create(ctypes.byref(h), int(device))
    if st != Q4LIN_OK:
        raise Q4LinError(st, "q4lin_create")
    return h.value


def q4lin_destroy(handle: int) -> int:
    return _lib.q4lin_destroy(handle)


def q4lin_run(handle, x, qweight, scales, bias, out, M, N, K, group_size, scale_dtype,
              stream) -> int:
    """Raw call: pointers and the stream are integers (0 / None for NULL)."""
    return _lib.q4lin_run(handle, x, qweight, scales, bias, out, M, N, K, group_size,
                          scale_dtype, stream)


def q4lin_run_grouped(handle, problems, stream) -> int:
    """problems: a sequence of q4lin_problem_t (or of 10-tuples in its field order)."""
    arr = (q4lin_problem_t * max(1, len(problems)))()
    for i, p in enumerate(problems):
        arr[i] = p if isinstance(p, q4lin_problem_t) else q4lin_problem_t(*p)
    return _lib.q4lin_run_grouped(handle, arr, len(problems), stream)


def q4lin_run_grouped_array(handle, array, count, stream) -> int:
    """Raw call with a prebuilt ctypes array of q4lin_problem_t (no per-call marshalling)."""
    return _lib.q4lin_run_grouped(handle, array, int(count), stream)


def q4lin_run_static_scratch(x, qweight, scales, bias, out, N, K, group_size, scale_dtype,
                             stream) -> int:
    """Raw call of the allocation-free decode GEMV (pointers and stream as integers)."""
    return _lib.q4lin_run_static_scratch(x, qweight, scales, bias, out, N, K, group_size,
                                         scale_dtype, stream)


def q4lin_run_backward_dx(handle, d_out, qweight, scales, d_x, M, N, K, group_size,
                          scale_dtype, stream) -> int:
    """Raw call: d_x[M,K] = d_out[M,N] @ dequant(W)[N,K] (pointers and stream as integers)."""
    return _lib.q4lin_run_backward_dx(handle, d_out, qweight, scales, d_x, M, N, K,
                                      group_size, scale_dtype, stream)


def q4lin_run_requant(handle, latent, scales, qweight, N, K, group_size, scale_dtype,
                      stream) -> int:
    """Raw call: packed codes of fp32 latents [N,K] with frozen scales (integers as pointers)."""
    return _lib.q4lin_run_requant(handle, latent, scales, qweight, N, K, group_size,
                                  scale_dtype, stream)


def q4lin_plan(handle, x, qweight, scales, bias, out, M, N, K, group_size, scale_dtype):
    """Returns (status, path)."""
    path = _i32(0)
    st = _lib.q4lin_plan(handle, x, qweight, scales, bias, out, M, N, K, group_size,
                         scale_dtype, ctypes.byref(path))
    return st, path.value


def q4lin_plan_kernel(handle, x, qweight, scales, bias, out, M, N, K, group_size,
                      scale_dtype):
    """Returns (status, kernel)."""
    kernel = _i32(0)
    st = _lib.q4lin_plan_kernel(handle, x, qweight, scales, bias, out, M, N, K, group_size,
                                scale_dtype, ctypes.byref(kernel))
    return st, kernel.value


def q4lin_set_option(handle, option: int, value: int) -> int:
    return _lib.q4lin_set_option(handle, int(option), int(value))


def q4lin_get_option(handle, option: int):
    v = _i64(0)
    st = _lib.q4lin_get_option(handle, int(option), ctypes.byref(v))
    return st, v.value


def q4lin_check_device_status(handle, stream):
    code = _i32(0)
    st = _lib.q4lin_check_device_status(handle, stream, ctypes.byref(code))
    return st, code.value


def q4lin_run_kv_append(handle, cache, args, stream) -> int:
    """cache: q4lin_kv_cache_t; args: q4lin_kv_append_t (pointers as integers)."""
    return _lib.q4lin_run_kv_append(handle, cache, args, stream)


def q4lin_run_attention(handle, cache, args, stream) -> int:
    """cache: q4lin_kv_cache_t; args: q4lin_attention_t."""
    return _lib.q4lin_run_attention(handle, cache, args, stream)


def q4lin_run_logprobs(handle, args, stream) -> int:
    """args: q4lin_logprobs_t."""
    return _lib.q4lin_run_logprobs(handle, args, stream)


def q4lin_run_logprobs_backward(handle, args, stream) -> int:
    """args: q4lin_logprobs_backward_t."""
    return _lib.q4lin_run_logprobs_backward(handle, args, stream)


def q4lin_run_kv4_append(handle, cache, args, stream) -> int:
    """cache: q4lin_kv_cache_t of 4-bit codes; args: q4lin_kv_append_t."""
    return _lib.q4lin_run_kv4_append(handle, cache, args, stream)


def q4lin_run_kv4_read(handle, cache, args, stream) -> int:
    """cache: q4lin_kv_cache_t of 4-bit codes; args: q4lin_kv_read_t."""
    return _lib.q4lin_run_kv4_read(handle, cache, args, stream)


def q4lin_run_kv4_attention(handle, cache, args, stream) -> int:
    """cache: q4lin_kv_cache_t of 4-bit codes; args: q4lin_attention_t."""
    return _lib.q4lin_run_kv4_attention(handle, cache, args, stream)


def q4lin_run_norm_rope(handle, args, stream) -> int:
    """args: q4lin_norm_rope_t."""
    return _lib.q4lin_run_norm_rope(handle, args, stream)


def q4lin_run_norm_rope_backward(handle, args, stream) -> int:
    """args: q4lin_norm_rope_backward_t."""
    return _lib.q4lin_run_norm_rope_backward(handle, args, stream)


# ---------------------------------------------------------------- torch convenience
class Handle:
    """Owns a q4lin handle for one CUDA device."""

    def __init__(self, device: int = 0):
        self.device = device
        self.ptr = q4lin_create(device)

    def close(self):
        if self.ptr:
            q4lin_destroy(self.ptr)
            self.ptr = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def set_option(self, option: int, value: int):
        st = q4lin_set_option(self.ptr, option, value)
        if st != Q4LIN_OK:
            raise Q4LinError(st, "q4lin_set_option")


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _check_args(x, qweight, scales, bias, group_size):
    import torch
    if x.dtype != torch.float32 or not x.is_contiguous() or x.dim() != 2:
        raise ValueError("x must be a contiguous float32 [M, K] tensor")
    M, K = x.shape
    if qweight.dtype != torch.uint8 or not qweight.is_contiguous() or qweight.dim() != 2 \
            or qweight.shape[1] != (K + 1) // 2:
        raise ValueError("qweight must be a contiguous uint8 [N, ceil(K/2)] tensor")
    N = qweight.shape[0]
    if scales.dtype == torch.float16:
        sd = Q4LIN_SCALE_F16
    elif scales.dtype == torch.float32:
        sd = Q4LIN_SCALE_F32
    else:
        raise ValueError("scales must be float32 or float16")
    if not scales.is_contiguous() or scales.numel() != -(-K // group_size) * N:
        raise ValueError("scales must be a contiguous [ceil(K/group_size), N] tensor")
    if bias is not None and (bias.dtype != torch.float32 or not bias.is_contiguous()
                             or bias.numel() != N):
        raise ValueError("bias must be a contiguous float32 [N] tensor or None")
    return M, N, K, sd


def _empty(shape, dtype, device, stream):
    """An output of a call on `stream` (a raw handle; None: the current stream).  Memory of the
    current stream may still be in use there, so on another one the output comes from that
    stream's, and is not given away before both are done with it."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    current = torch.cuda.current_stream(device)
    if stream == current.cuda_stream:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=device)):
        out = torch.empty(shape, dtype=dtype, device=device)
    out.record_stream(current)
    return out


def linear(handle: Handle, x, qweight, scales, bias, group_size: int, out=None,
           stream=None):
    """out[M,N] = x @ dequant(qweight)^T (+ bias) on the current (or given) stream; another
    stream's inputs have to be ready there, and kept until it has read them."""
    import torch
    M, N, K, sd = _check_args(x, qweight, scales, bias, group_size)
    if out is None:
        out = _empty((M, N), torch.float32, x.device, stream)
    s = stream if stream is not None else torch.cuda.current_stream(x.device).cuda_stream
    st = q4lin_run(handle.ptr, _ptr(x), _ptr(qweight), _ptr(scales), _ptr(bias),
                   _ptr(out), M, N, K, group_size, sd, s)
    if st != Q4LIN_OK:
        raise Q4LinError(st, "q4lin_run")
    return out


def plan(handle: Handle, x, qweight, scales, bias, group_size: int, out) -> str:
    """Name of the kernel family q4lin_run would use for these tensors."""
    M, N, K, sd = _check_args(x, qweight, scales, bias, group_size)
    st, path = q4lin_plan(handle.ptr, _ptr(x), _ptr(qweight), _ptr(scales), _ptr(bias),
                          _ptr(out), M, N, K, group_size, sd)
    if st != Q4LIN_OK:
        raise Q4LinError(st, "q4lin_plan")
    return PATH_NAMES[path]


def plan_kernel(handle: Handle, x, qweight, scales, bias, group_size: int, out) -> str:
    """Name of the kernel q4lin_run would launch for these tensors."""
    M, N, K, sd = _check_args(x, qweight, scales, bias, group_size)
    st, kernel = q4lin_plan_kernel(handle.ptr, _ptr(x), _ptr(qweight), _ptr(scales),
                                   _ptr(bias), _ptr(out), M, N, K, group_size, sd)
    if st != Q4LIN_OK:
        raise Q4LinError(st, "q4lin_plan_kernel")
    return KERNEL_NAMES[kernel]


# ------------------------------------------------- operators around the linears (torch)
# A decode step makes hundreds of these calls, some shorter on the GPU than their checks
# here: types are compared as objects, and torch is looked up once.
# `stream` is a raw handle (default: torch's current stream).  On another stream than theirs,
# inputs have to be ready there, and kept until it has read them.  None of these calls is seen by
# autograd: gradients are calls of their own (logprobs_backward, q4lin_run_backward_dx).
class _Torch:
    """torch, its types' codes and its current stream's handle, filled at the first use."""
    module = None
    codes: dict = {}

    @classmethod
    def load(cls):
        import torch
        cls.float32, cls.int32, cls.empty = torch.float32, torch.int32, torch.empty
        cls.codes = {torch.float32: Q4LIN_DTYPE_F32, torch.float16: Q4LIN_DTYPE_F16,
                     torch.bfloat16: Q4LIN_DTYPE_BF16}
        # The raw handle without a Stream object around it, where torch has that.
        cls.stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
            (lambda device: torch.cuda.current_stream(device).cuda_stream)
        cls.module = torch


def _dtype_code(t, what):
    code = _Torch.codes.get(t.dtype)
    if code is None:
        raise ValueError(f"{what} must be float32, float16 or bfloat16")
    return code


def _check_device(handle, *tensors):
    if _Torch.module is None:
        _Torch.load()
    device = handle.device
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise ValueError(f"every tensor must be on the handle's device, cuda:{device}")


def _check_vector(t, n, dtype, what):
    """A contiguous one-dimensional tensor of n values."""
    if t.dtype is not dtype or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} [{n}] tensor")
    return t.data_ptr()


def _head_strides(t, what):
    """Token and head strides of [tokens, heads, head_dim] with contiguous channels."""
    strides = t.stride()
    if len(strides) != 3 or (strides[2] != 1 and t.numel()):
        raise ValueError(f"{what} must be [tokens, heads, head_dim] with contiguous channels")
    return strides


def _new(shape, dtype, device, stream):
    if stream is None:
        return _Torch.empty(shape, dtype=dtype, device=device)
    return _empty(shape, dtype, device, stream)


def _stream_of(stream, handle) -> int:
    if stream is not None:
        return stream
    return _Torch.stream(handle.device)


def _rope_members(cos, sin, interleaved):
    """The members of q4lin_rope_t."""
    shape, float32 = cos.shape, _Torch.float32
    if cos.dtype is not float32 or sin.dtype is not float32 or len(shape) != 2 \
            or sin.shape != shape or not cos.is_contiguous() or not sin.is_contiguous():
        raise ValueError("rope must be two contiguous float32 [positions, rotated / 2] tensors")
    return cos.data_ptr(), sin.data_ptr(), shape[0], 2 * shape[1], interleaved


def _rope_args(rope, interleaved):
    if rope is None:
        return q4lin_rope_t()
    return q4lin_rope_t(*_rope_members(*rope, interleaved))


class _PagedCache:
    """What the paged caches share: `shapes` gives the codes' and scales' shapes."""

    def __init__(self, k_codes, k_scales, v_codes, v_scales, page_table):
        pages, heads, page, dim = self.sizes(k_codes)
        shapes = self.shapes(pages, heads, page, dim)
        for t, shape, kind, what in zip((k_codes, v_codes, k_scales, v_scales), shapes,
                                        ("uint8", "uint8", "float32", "float32"),
                                        ("k_codes", "v_codes", "k_scales", "v_scales")):
            if tuple(t.shape) != shape or str(t.dtype) != "torch." + kind or not t.is_contiguous():
                raise ValueError(f"{what} must be a contiguous {kind} {list(shape)} tensor")
        if page_table.dim() != 2 or str(page_table.dtype) != "torch.int32" or \
                (page_table.shape[1] > 1 and page_table.stride(1) != 1):
            raise ValueError("page_table must be an int32 [batch, pages] tensor with contiguous rows")
        if len({t.device for t in (k_codes, k_scales, v_codes, v_scales, page_table)}) != 1:
            raise ValueError("a cache's tensors must be on one device")
        self.k_codes, self.k_scales = k_codes, k_scales
        self.v_codes, self.v_scales = v_codes, v_scales
        self.page_table = page_table
        batch, width = page_table.shape
        stride = page_table.stride(0) if batch > 1 else width
        self.args = q4lin_kv_cache_t(k_codes.data_ptr(), k_scales.data_ptr(), v_codes.data_ptr(),
                                     v_scales.data_ptr(), page_table.data_ptr(), pages, heads, page,
                                     dim, batch, width, stride)

    @classmethod
    def empty(cls, num_pages: int, kv_heads: int, page_size: int, head_dim: int, page_table):
        """A cache with nothing in it, on the page table's device."""
        import torch
        k, v, ks, vs = cls.shapes(num_pages, kv_heads, page_size, head_dim)
        codes = lambda shape: torch.full(shape, cls.zero, dtype=torch.uint8, device=page_table.device)
        scales = lambda shape: torch.zeros(shape, device=page_table.device)
        return cls(codes(k), scales(ks), codes(v), scales(vs), page_table)


class KVCache(_PagedCache):
    """The tensors of a paged 8-bit key/value cache (q4lin_kv_cache_t).

    k_codes uint8 [num_pages, kv_heads, page_size, head_dim], v_codes uint8 [num_pages,
    kv_heads, head_dim, page_size], k_scales and v_scales float32 [num_pages, kv_heads],
    page_table int32 [batch, pages per sequence].  The tensors stay the caller's; the page
    table's contents may change between calls."""
    zero = 128  # the bytes that stand for 0
    run_append, run_attention = _lib.q4lin_run_kv_append, _lib.q4lin_run_attention

    @staticmethod
    def sizes(k_codes):
        if k_codes.dim() != 4:
            raise ValueError("k_codes must be [num_pages, kv_heads, page_size, head_dim]")
        return tuple(k_codes.shape)

    @staticmethod
    def shapes(pages, heads, page, dim):
        return ((pages, heads, page, dim), (pages, heads, dim, page), (pages, heads), (pages, heads))


class KVCache4(_PagedCache):
    """The tensors of a paged 4-bit key/value cache (q4lin_kv4_cache_t), for kv_append, kv_read
    and attention.

    k_codes and v_codes uint8 [num_pages, kv_heads, page_size, head_dim / 2] (the even channel
    in the low four bits), k_scales and v_scales float32 [num_pages, kv_heads, page_size],
    page_table as in KVCache."""
    zero = 0x88
    run_append, run_attention = _lib.q4lin_run_kv4_append, _lib.q4lin_run_kv4_attention

    @staticmethod
    def sizes(k_codes):
        if k_codes.dim() != 4:
            raise ValueError("k_codes must be [num_pages, kv_heads, page_size, head_dim / 2]")
        pages, heads, page, half = k_codes.shape
        return pages, heads, page, 2 * half

    @staticmethod
    def shapes(pages, heads, page, dim):
        if dim % 2:
            raise ValueError("head_dim must be even")
        codes, scales = (pages, heads, page, dim // 2), (pages, heads, page)
        return codes, codes, scales, scales


def kv_append(handle: Handle, cache, k, v, offsets, starts, rope=None,
              interleaved: bool = False, stream=None) -> None:
    """Append k (rotated by rope = (cos, sin) on the way) and v, [tokens, kv_heads, head_dim]
    each and possibly slices of a larger tensor, to the cache (KVCache or KVCache4): rows
    offsets[b] .. offsets[b + 1] become tokens starts[b], starts[b] + 1, ... of sequence b."""
    c = cache.args
    cos, sin = rope or (None, None)
    _check_device(handle, cache.k_codes, k, v, offsets, starts, cos, sin)
    ks, vs, shape = _head_strides(k, "k"), _head_strides(v, "v"), k.shape
    if v.shape != shape or shape[1] != c.kv_heads or shape[2] != c.head_dim or v.dtype is not k.dtype:
        raise ValueError("k and v must be [tokens, kv_heads, head_dim] of one type, as the cache")
    batch, int32 = c.batch, _Torch.int32
    args = q4lin_kv_append_t(k.data_ptr(), v.data_ptr(), ks[0], ks[1], vs[0], vs[1],
                             _dtype_code(k, "k"), shape[0],
                             _check_vector(offsets, batch + 1, int32, "offsets"),
                             _check_vector(starts, batch, int32, "starts"),
                             _rope_args(rope, interleaved))
    run = cache.run_append
    st = run(handle.ptr, c, args, _stream_of(stream, handle))
    if st != Q4LIN_OK:
        raise Q4LinError(st, run.__name__)


def kv_read(handle: Handle, cache: KVCache4, offsets, starts, tokens: int, dtype=None, k=None,
            v=None, stream=None):
    """Tokens of a 4-bit cache as dense keys and values [tokens, kv_heads, head_dim] of `dtype`
    (default float32): token starts[b] + i of sequence b becomes row offsets[b] + i; `tokens` rows
    in all.  k and v: outputs to use (rows of no sequence are left as they are there)."""
    c = cache.args
    if not isinstance(cache, KVCache4):
        raise ValueError("cache must be a KVCache4")
    _check_device(handle, cache.k_codes, offsets, starts, k, v)
    given = k if k is not None else v
    if dtype is None:
        dtype = _Torch.float32 if given is None else given.dtype
    code = _Torch.codes.get(dtype)
    if code is None:
        raise ValueError("dtype must be float32, float16 or bfloat16")
    shape = tokens, c.kv_heads, c.head_dim
    for t, what in ((k, "k"), (v, "v")):
        if t is not None and (t.shape != shape or t.dtype is not dtype or not t.is_contiguous()):
            raise ValueError(f"{what} must be a contiguous {dtype} {list(shape)} tensor")
    device = cache.k_codes.device
    k = _new(shape, dtype, device, stream) if k is None else k
    v = _new(shape, dtype, device, stream) if v is None else v
    batch, int32 = c.batch, _Torch.int32
    args = q4lin_kv_read_t(k.data_ptr(), v.data_ptr(), code, tokens,
                           _check_vector(offsets, batch + 1, int32, "offsets"),
                           _check_vector(starts, batch, int32, "starts"))
    st = _lib.q4lin_run_kv4_read(handle.ptr, c, args, _stream_of(stream, handle))
    if st != Q4LIN_OK:
        raise Q4LinError(st, "q4lin_run_kv4_read")
    return k, v


def attention(handle: Handle, cache, query, offsets, lengths, scale: float,
              max_query: Optional[int] = None, rope=None, interleaved: bool = False,
              causal: bool = True, window: int = 0, out=None, lse=None, stream=None):
    """Attention of query [tokens, heads, head_dim] over the cache (q4lin_run_attention, or
    q4lin_run_kv4_attention for a KVCache4).
    lengths[b] counts sequence b's tokens in the cache, those of its queries included;
    max_query: no sequence has more query tokens (default: all of them; 1 for single tokens
    spares a batch the launches for prompts).  Returns (out, lse): out like query, lse float32
    [tokens, heads]."""
    c = cache.args
    cos, sin = rope or (None, None)
    _check_device(handle, cache.k_codes, query, offsets, lengths, out, lse, cos, sin)
    strides, shape = _head_strides(query, "query"), query.shape
    tokens, heads, dim = shape
    if dim != c.head_dim or heads % c.kv_heads:
        raise ValueError("query must be [tokens, heads, head_dim], heads a multiple of kv_heads")
    if out is None:
        out = _new(shape, query.dtype, query.device, stream)
    elif out.shape != shape or out.dtype is not query.dtype or not out.is_contiguous():
        raise ValueError("out must be contiguous, with the query's shape and type")
    if lse is None:
        lse = _new((tokens, heads), _Torch.float32, query.device, stream)
    elif lse.shape != (tokens, heads) or lse.dtype is not _Torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 [tokens, heads] tensor")
    batch, int32 = c.batch, _Torch.int32
    args = q4lin_attention_t(query.data_ptr(), strides[0], strides[1], out.data_ptr(),
                             lse.data_ptr(), _dtype_code(query, "query"), tokens, heads,
                             tokens if max_query is None else max_query,
                             _check_vector(offsets, batch + 1, int32, "offsets"),
                             _check_vector(lengths, batch, int32, "lengths"), scale,
                             causal, window, _rope_args(rope, interleaved))
    run = cache.run_attention
    st = run(handle.ptr, c, args, _stream_of(stream, handle))
    if st != Q4LIN_OK:
        raise Q4LinError(st, run.__name__)
    return out, lse


# q4lin_norm_rope_t and what q4lin_norm_rope_backward_t has behind it, packed: a ctypes structure of
# as many members takes five times as long to fill as these calls' kernels to launch.
_NORM_ROPE = struct.Struct("PPqqqqPPPPqqqqi4xqqqqPPPqqi4xf4x")
_NORM_ROPE_MORE = struct.Struct("PPqqqqPP")
_run_norm_rope = _lib["q4lin_run_norm_rope"]
_run_norm_rope_backward = _lib["q4lin_run_norm_rope_backward"]
for _f, _t in ((_run_norm_rope, q4lin_norm_rope_t), (_run_norm_rope_backward, q4lin_norm_rope_backward_t)):
    _f.argtypes, _f.restype = [_vp, ctypes.c_char_p, _vp], _i32
assert _NORM_ROPE.size == ctypes.sizeof(q4lin_norm_rope_t)
assert _NORM_ROPE.size + _NORM_ROPE_MORE.size == ctypes.sizeof(q4lin_norm_rope_backward_t)


def _norm_args(handle, q, k, q_weight, k_weight, positions, rope, eps, interleaved, q_out, k_out,
               stream):
    """(a packed q4lin_norm_rope_t, q_out, k_out); the outputs are made where they are not given."""
    cos, sin = rope if rope is not None else (None, None)
    _check_device(handle, q, k, q_weight, k_weight, positions, cos, sin, q_out, k_out)
    qs, ks = _head_strides(q, "q"), _head_strides(k, "k")
    q_shape, k_shape, dtype = q.shape, k.shape, q.dtype
    tokens, heads, dim = q_shape
    if k_shape[0] != tokens or k_shape[2] != dim or k.dtype is not dtype:
        raise ValueError("q and k must be [tokens, heads, head_dim] and [tokens, kv_heads, head_dim] of one type")
    code = _dtype_code(q, "q")
    if q_out is None:
        q_out = _new(q_shape, dtype, q.device, stream)
    elif q_out.shape != q_shape or q_out.dtype is not dtype:
        raise ValueError("the output for q must have its shape and type")
    if k_out is None:
        k_out = _new(k_shape, dtype, k.device, stream)
    elif k_out.shape != k_shape or k_out.dtype is not dtype:
        raise ValueError("the output for k must have its shape and type")
    qos, kos = _head_strides(q_out, "the output for q"), _head_strides(k_out, "the output for k")
    float32 = _Torch.float32
    qw = 0 if q_weight is None else _check_vector(q_weight, dim, float32, "q_weight")
    kw = 0 if k_weight is None else _check_vector(k_weight, dim, float32, "k_weight")
    at = 0 if positions is None else _check_vector(positions, tokens, _Torch.int32, "positions")
    if rope is None:
        turn = 0, 0, 0, 0, 0
    elif positions is None:
        raise ValueError("a rotation needs positions")
    else:
        turn = _rope_members(cos, sin, interleaved)
    args = _NORM_ROPE.pack(q.data_ptr(), k.data_ptr(), qs[0], qs[1], ks[0], ks[1], qw, kw,
                           q_out.data_ptr(), k_out.data_ptr(), qos[0], qos[1], kos[0], kos[1], code,
                           tokens, heads, k_shape[1], dim, at, *turn, eps)
    return args, q_out, k_out


def norm_rope(handle: Handle, q, k, q_weight=None, k_weight=None, positions=None, rope=None,
              eps: float = 1e-6, interleaved: bool = False, q_out=None, k_out=None, stream=None):
    """q [tokens, heads, head_dim] and k [tokens, kv_heads, head_dim], possibly slices of a larger
    tensor, normalised per head, times their weights (float32 [head_dim], None for ones), and
    rotated by rope = (cos, sin) at positions (int32 [tokens]).  q_out and k_out: outputs to use,
    q and k themselves among them.  Returns (q_out, k_out)."""
    args, q_out, k_out = _norm_args(handle, q, k, q_weight, k_weight, positions, rope, eps,
                                    interleaved, q_out, k_out, stream)
    st = _run_norm_rope(handle.ptr, args, _stream_of(stream, handle))
    if st != Q4LIN_OK:
        raise Q4LinError(st, "q4lin_run_norm_rope")
    return q_out, k_out


class NormRopeGradients(NamedTuple):
    """Results of norm_rope_backward: like q and k, and float32 [head_dim] each (None where the
    weight was None)."""
    d_q: object
    d_k: object
    d_q_weight: object
    d_k_weight: object


def norm_rope_backward(handle: Handle, q, k, q_weight, k_weight, positions, rope, d_q_out, d_k_out,
                       eps: float = 1e-6, interleaved: bool = False, d_q=None, d_k=None,
                       stream=None) -> NormRopeGradients:
    """Gradients of norm_rope for q, k and the weights, given its inputs and the gradients for
    its outputs (of any token and head strides).  d_q and d_k: outputs to use; d_q may be q or d_q_out, d_k may be
    k or d_k_out."""
    forward, d_q, d_k = _norm_args(handle, q, k, q_weight, k_weight, positions, rope, eps,
                                   interleaved, d_q, d_k, stream)
    _check_device(handle, d_q_out, d_k_out)
    if d_q_out.shape != q.shape or d_k_out.shape != k.shape or d_q_out.dtype is not q.dtype \
            or d_k_out.dtype is not q.dtype:
        raise ValueError("d_q_out and d_k_out must have the shapes and the type of q and k")
    dqs, dks = _head_strides(d_q_out, "d_q_out"), _head_strides(d_k_out, "d_k_out")
    dqw = None if q_weight is None else _new(q_weight.shape, _Torch.float32, q.device, stream)
    dkw = None if k_weight is None else _new(k_weight.shape, _Torch.float32, q.device, stream)
    args = forward + _NORM_ROPE_MORE.pack(d_q_out.data_ptr(), d_k_out.data_ptr(), dqs[0], dqs[1], dks[0],
                                          dks[1], 0 if dqw is None else dqw.data_ptr(),
                                          0 if dkw is None else dkw.data_ptr())
    st = _run_norm_rope_backward(handle.ptr, args, _stream_of(stream, handle))
    if st != Q4LIN_OK:
        raise Q4LinError(st, "q4lin_run_norm_rope_backward")
    return NormRopeGradients(d_q, d_k, dqw, dkw)


class LogProbs(NamedTuple):
    """Results of logprobs: float32 [rows] each; the top alternatives (None without any) as
    int32 and float32 [rows, top], largest first."""
    logprob: object
    entropy: object
    lse: object
    top_tokens: object
    top_logprobs: object


def _row_stride(t, what):
    strides = t.stride()
    if len(strides) != 2 or (strides[1] != 1 and t.shape[1] != 1):
        raise ValueError(f"{what} must be [rows, vocabulary] with contiguous rows")
    return strides[0] if t.shape[0] > 1 else t.shape[1]  # (one row's may be anything)


def logprobs(handle: Handle, logits, tokens=None, top: int = 0, stream=None) -> LogProbs:
    """Log probability of tokens (int32 [rows], -1 for none), entropy, log-sum-exp and the
    `top` most likely tokens of each row of logits (q4lin_run_logprobs)."""
    _check_device(handle, logits, tokens)
    stride = _row_stride(logits, "logits")
    rows, vocabulary = logits.shape
    device, float32 = logits.device, _Torch.float32
    logprob, entropy, lse = (_new(rows, float32, device, stream) for _ in range(3))
    ids = best = None
    if top:
        ids = _new((rows, top), _Torch.int32, device, stream)
        best = _new((rows, top), float32, device, stream)
    args = q4lin_logprobs_t(
        logits.data_ptr(), stride, _dtype_code(logits, "logits"), rows, vocabulary,
        None if tokens is None else _check_vector(tokens, rows, _Torch.int32, "tokens"),
        logprob.data_ptr(), entropy.data_ptr(), lse.data_ptr(), top, _ptr(ids), _ptr(best))
    st = _lib.q4lin_run_logprobs(handle.ptr, args, _stream_of(stream, handle))
    if st != Q4LIN_OK:
        raise Q4LinError(st, "q4lin_run_logprobs")
    return LogProbs(logprob, entropy, lse, ids, best)


def logprobs_backward(handle: Handle, logits, tokens, lse, entropy, d_logprob=None,
                      d_entropy=None, out=None, stream=None):
    """Gradient for the logits of logprobs' logprob and entropy, given theirs (float32 [rows]
    or None for zeros) and the lse and entropy that logprobs returned.  out may be the logits
    themselves."""
    _check_device(handle, logits, tokens, lse, entropy, d_logprob, d_entropy, out)
    stride = _row_stride(logits, "logits")
    rows, vocabulary = logits.shape
    if out is None:
        out = _new((rows, vocabulary), logits.dtype, logits.device, stream)
    elif out.shape != logits.shape or out.dtype is not logits.dtype:
        raise ValueError("out must have the logits' shape and type")
    float32 = _Torch.float32
    vector = lambda t, what: None if t is None else _check_vector(t, rows, float32, what)
    args = q4lin_logprobs_backward_t(
        logits.data_ptr(), stride, _dtype_code(logits, "logits"), rows, vocabulary,
        None if tokens is None else _check_vector(tokens, rows, _Torch.int32, "tokens"),
        vector(lse, "lse"), vector(entropy, "entropy"), vector(d_logprob, "d_logprob"),
        vector(d_entropy, "d_entropy"), out.data_ptr(), _row_stride(out, "out"))
    st = _lib.q4lin_run_logprobs_backward(handle.ptr, args, _stream_of(stream, handle))
    if st != Q4LIN_OK:
        raise Q4LinError(st, "q4lin_run_logprobs_backward")
    return out
