"""Python binding of the GB300 packed quantized-weight decoder (``libndq.so``).

Argument marshalling only: every decode step runs in the library's CUDA
kernels.  The ``ndq_*`` functions mirror the C ABI in ``include/ndq.h`` one
to one (plain integers and pointers); ``dequantize_packed``,
``dequantize_packed_batched``, ``matmul_packed``, ``kv_plan``, ``kv_append``,
``attention_kv8``, ``lora_add`` and the like are conveniences that take torch
CUDA tensors and the current torch stream.  There is no CPU fallback: importing this
module fails if the library has not been built
(``python -m quantized_weight_block_gb300.build``).
"""
from __future__ import annotations

import ctypes
import os

from . import build as _build

LIB_PATH = _build.LIB

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python -m quantized_weight_block_gb300.build` "
                      "(there is no CPU fallback)")

_lib = ctypes.CDLL(LIB_PATH)

# ---- constants mirrored from include/ndq.h --------------------------------
NDQ_OK = 0
STATUS = {
    0: "NDQ_OK", 1: "NDQ_ERR_NULL", 2: "NDQ_ERR_UNKNOWN_FORMAT", 3: "NDQ_ERR_UNSUPPORTED_FORMAT",
    4: "NDQ_ERR_BAD_RANK", 5: "NDQ_ERR_NEGATIVE_DIM", 6: "NDQ_ERR_NOT_BLOCK_ALIGNED",
    7: "NDQ_ERR_LENGTH_MISMATCH", 8: "NDQ_ERR_OVERFLOW", 9: "NDQ_ERR_BAD_DTYPE", 10: "NDQ_ERR_WORKSPACE",
    11: "NDQ_ERR_CUDA", 12: "NDQ_ERR_DEVICE_FAULT", 13: "NDQ_ERR_BAD_COUNT", 14: "NDQ_ERR_TOO_MANY_TENSORS",
    15: "NDQ_ERR_BAD_ARG", 16: "NDQ_ERR_MISALIGNED",
}
NDQ_FLOAT, NDQ_FLOAT16, NDQ_DOUBLE, NDQ_BFLOAT16 = 1, 10, 11, 16
NDQ_INT8, NDQ_FLOAT8E4M3FN = 3, 17
NDQ_MAX_RANK = 8
NDQ_NUM_FORMATS = 36
NDQ_NOALLOC_MAX_TENSORS = 1024


class NdqError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        self.name = STATUS.get(status, str(status))
        msg = _lib.ndq_status_string(status).decode()
        super().__init__(f"{self.name}: {msg}" + (f" ({what})" if what else ""))


class ndq_tensor_desc(ctypes.Structure):
    _fields_ = [
        ("format_id", ctypes.c_int32), ("ndim", ctypes.c_int32), ("shape", ctypes.c_int64 * NDQ_MAX_RANK),
        ("out_dtype", ctypes.c_int32), ("reserved", ctypes.c_int32), ("x", ctypes.c_void_p),
        ("x_len", ctypes.c_uint64), ("y", ctypes.c_void_p),
    ]


class ndq_matmul_desc(ctypes.Structure):
    _fields_ = [
        ("format_id", ctypes.c_int32), ("reserved", ctypes.c_int32), ("n", ctypes.c_int64), ("w", ctypes.c_void_p),
        ("w_len", ctypes.c_uint64), ("y", ctypes.c_void_p),
    ]


class ndq_kv_cache(ctypes.Structure):
    _fields_ = [
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
        ("num_blocks", ctypes.c_int64), ("kv_heads", ctypes.c_int32), ("block_size", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("code_type", ctypes.c_int32),
    ]


_c = ctypes
_lib.ndq_format_from_name.argtypes = [_c.c_char_p]
_lib.ndq_format_from_name.restype = _c.c_int
_lib.ndq_format_name.argtypes = [_c.c_int]
_lib.ndq_format_name.restype = _c.c_char_p
_lib.ndq_format_geometry.argtypes = [_c.c_int, _c.POINTER(_c.c_int), _c.POINTER(_c.c_int)]
_lib.ndq_format_supported.argtypes = [_c.c_int]
_lib.ndq_status_string.argtypes = [_c.c_int]
_lib.ndq_status_string.restype = _c.c_char_p
_lib.ndq_payload_geometry.argtypes = [_c.c_int, _c.POINTER(_c.c_int64), _c.c_int, _c.c_uint64,
                                      _c.POINTER(_c.c_uint64), _c.POINTER(_c.c_uint64), _c.POINTER(_c.c_uint64)]
_lib.ndq_dequantize_packed.argtypes = [_c.c_int, _c.POINTER(_c.c_int64), _c.c_int, _c.c_int, _c.c_void_p,
                                       _c.c_size_t, _c.c_void_p, _c.c_void_p]
_lib.ndq_batched_workspace_bytes.argtypes = [_c.c_int]
_lib.ndq_batched_workspace_bytes.restype = _c.c_size_t
_lib.ndq_dequantize_packed_batched.argtypes = [_c.POINTER(ndq_tensor_desc), _c.c_int, _c.c_void_p, _c.c_size_t,
                                               _c.c_void_p]
_lib.ndq_get_device_fault.argtypes = [_c.POINTER(_c.c_uint32)]
_lib.ndq_test_withhold_copy.argtypes = [_c.c_int64, _c.c_uint32]
_lib.ndq_test_lose_copies.argtypes = [_c.c_uint32]
_lib.ndq_dequantize_packed_batched_noalloc.argtypes = [_c.POINTER(ndq_tensor_desc), _c.c_int, _c.c_void_p]
_lib.ndq_matmul_packed.argtypes = [_c.c_int, _c.c_int64, _c.c_int64, _c.c_void_p, _c.c_size_t, _c.c_void_p,
                                   _c.c_int64, _c.c_int, _c.c_int, _c.c_void_p, _c.c_void_p]
_lib.ndq_matmul_packed_batched.argtypes = [_c.POINTER(ndq_matmul_desc), _c.c_int, _c.c_int64, _c.c_void_p,
                                           _c.c_int64, _c.c_int, _c.c_int, _c.c_void_p]
_p, _i64 = _c.c_void_p, _c.c_int64
_lib.ndq_kv_plan.argtypes = [_p, _p, _i64, _c.c_int, _p, _p, _p, _i64, _p, _p, _p, _p, _i64, _p, _p]
_lib.ndq_kv_append.argtypes = [_c.POINTER(ndq_kv_cache), _p, _p, _c.c_int, _i64, _i64, _p, _i64, _p]
_lib.ndq_attention_workspace_bytes.argtypes = [_c.c_int]
_lib.ndq_attention_workspace_bytes.restype = _c.c_size_t
_lib.ndq_attention_kv8.argtypes = [_c.POINTER(ndq_kv_cache), _p, _c.c_int, _i64, _c.c_int, _i64, _p, _i64, _p, _p, _i64,
                                   _i64, _c.c_float, _i64, _p, _p, _p, _c.c_size_t, _p]
_lib.ndq_lora_workspace_bytes.argtypes = [_i64, _i64, _i64]
_lib.ndq_lora_workspace_bytes.restype = _c.c_size_t
_lib.ndq_lora_add.argtypes = [_p, _i64, _i64, _p, _p, _i64, _i64, _i64, _p, _p, _p, _p, _c.c_int, _p, _p, _c.c_size_t,
                              _p]

# Every symbol the header declares (checked by the CPU tests).
EXPORTS = (
    "ndq_format_from_name", "ndq_format_name", "ndq_format_geometry", "ndq_format_supported",
    "ndq_status_string", "ndq_payload_geometry", "ndq_dequantize_packed", "ndq_batched_workspace_bytes",
    "ndq_dequantize_packed_batched", "ndq_get_device_fault", "ndq_dequantize_packed_batched_noalloc",
    "ndq_matmul_packed", "ndq_test_withhold_copy", "ndq_matmul_packed_batched",
    "ndq_kv_plan", "ndq_kv_append", "ndq_attention_workspace_bytes", "ndq_attention_kv8",
    "ndq_lora_workspace_bytes", "ndq_lora_add", "ndq_test_lose_copies",
)


# ---- raw C ABI (same names, plain integers / pointers) --------------------
def ndq_format_from_name(name: str) -> int:
    return _lib.ndq_format_from_name(name.encode() if name is not None else None)


def ndq_format_name(format_id: int) -> str | None:
    r = _lib.ndq_format_name(format_id)
    return r.decode() if r is not None else None


def ndq_format_geometry(format_id: int) -> tuple[int, int]:
    B, S = _c.c_int(), _c.c_int()
    rc = _lib.ndq_format_geometry(format_id, _c.byref(B), _c.byref(S))
    if rc:
        raise NdqError(rc)
    return B.value, S.value


def ndq_format_supported(format_id: int) -> int:
    return _lib.ndq_format_supported(format_id)


def ndq_status_string(status: int) -> str:
    return _lib.ndq_status_string(status).decode()


def _shape(shape):
    s = [int(d) for d in shape]
    return (_c.c_int64 * max(1, len(s)))(*s), len(s)


def ndq_payload_geometry(format_id: int, shape, x_len: int) -> tuple[int, int, int]:
    sa, nd = _shape(shape)
    nb, ne, ndv = _c.c_uint64(), _c.c_uint64(), _c.c_uint64()
    rc = _lib.ndq_payload_geometry(format_id, sa, nd, x_len, _c.byref(nb), _c.byref(ne), _c.byref(ndv))
    if rc:
        raise NdqError(rc)
    return nb.value, ne.value, ndv.value


def ndq_dequantize_packed(format_id: int, shape, out_dtype: int, x_ptr: int, x_len: int, y_ptr: int,
                          stream: int = 0) -> int:
    """Raw call; returns the status code (0 on success)."""
    sa, nd = _shape(shape)
    return _lib.ndq_dequantize_packed(format_id, sa, nd, out_dtype, x_ptr, x_len, y_ptr, stream)


def ndq_batched_workspace_bytes(n: int) -> int:
    return _lib.ndq_batched_workspace_bytes(n)


def ndq_dequantize_packed_batched(descs, workspace_ptr: int, ws_bytes: int, stream: int = 0) -> int:
    """Raw call over a sequence of ndq_tensor_desc; returns the status code."""
    arr = (ndq_tensor_desc * max(1, len(descs)))(*descs)
    return _lib.ndq_dequantize_packed_batched(arr, len(descs), workspace_ptr, ws_bytes, stream)


def ndq_dequantize_packed_batched_noalloc(descs, stream: int = 0) -> int:
    """Raw call of the no-allocation batched decode (launch table held in the
    library's own device array); returns the status code."""
    arr = (ndq_tensor_desc * max(1, len(descs)))(*descs)
    return _lib.ndq_dequantize_packed_batched_noalloc(arr, len(descs), stream)


def ndq_matmul_packed(format_id: int, N: int, K: int, w_ptr: int, w_len: int, x_ptr: int, M: int,
                      weight_dtype: int, out_dtype: int, y_ptr: int, stream: int = 0) -> int:
    """Raw call of the fused decode + product; returns the status code."""
    return _lib.ndq_matmul_packed(format_id, N, K, w_ptr, w_len, x_ptr, M, weight_dtype, out_dtype, y_ptr, stream)


def ndq_matmul_packed_batched(descs, K: int, x_ptr: int, M: int, weight_dtype: int, out_dtype: int,
                              stream: int = 0) -> int:
    """Raw call over a sequence of ndq_matmul_desc sharing X; returns the status code."""
    arr = (ndq_matmul_desc * max(1, len(descs)))(*descs)
    return _lib.ndq_matmul_packed_batched(arr, len(descs), K, x_ptr, M, weight_dtype, out_dtype, stream)


def ndq_test_withhold_copy(tile: int, wait_limit_us: int) -> int:
    """Raw call: the next decode launch of this host thread withholds one
    tile's staging copy (a check of the device-side failure path); returns
    the status code."""
    return _lib.ndq_test_withhold_copy(tile, wait_limit_us)


def ndq_test_lose_copies(wait_limit_us: int) -> int:
    """Raw call: the next attention or adapter launch of this host thread sees
    none of its staged copies land (a check of the device-side failure path);
    returns the status code."""
    return _lib.ndq_test_lose_copies(wait_limit_us)


def ndq_get_device_fault() -> int:
    v = _c.c_uint32()
    rc = _lib.ndq_get_device_fault(_c.byref(v))
    if rc:
        raise NdqError(rc)
    return v.value


# ---- torch conveniences ----------------------------------------------------
def _torch():
    import torch
    return torch


def out_dtype_code(dtype) -> int:
    torch = _torch()
    return {torch.float32: NDQ_FLOAT, torch.float16: NDQ_FLOAT16, torch.bfloat16: NDQ_BFLOAT16,
            torch.float64: NDQ_DOUBLE}[dtype]


def format_id(fmt) -> int:
    if isinstance(fmt, int):
        return fmt
    i = ndq_format_from_name(fmt)
    if i < 0:
        raise NdqError(2, str(fmt))
    return i


def _stream_handle(stream) -> int:
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return int(s.cuda_stream)


def dequantize_packed(fmt, shape, x, out_dtype=None, y=None, stream=None):
    """Decode one payload held in a CUDA uint8 tensor; returns y (shape `shape`)."""
    torch = _torch()
    out_dtype = out_dtype or torch.float32
    if y is None:
        y = torch.empty(tuple(int(s) for s in shape), dtype=out_dtype, device=x.device)
    if x.dtype != torch.uint8 or not x.is_contiguous() or not y.is_contiguous():
        raise ValueError("x must be a contiguous uint8 tensor and y contiguous")
    rc = ndq_dequantize_packed(format_id(fmt), shape, out_dtype_code(y.dtype), x.data_ptr(), x.numel(),
                               y.data_ptr(), _stream_handle(stream))
    if rc:
        raise NdqError(rc, str(fmt))
    return y


def make_desc(fmt, shape, x, y) -> ndq_tensor_desc:
    d = ndq_tensor_desc()
    d.format_id = format_id(fmt)
    d.ndim = len(shape)
    for i, s in enumerate(shape):
        d.shape[i] = int(s)
    d.out_dtype = out_dtype_code(y.dtype)
    d.reserved = 0
    d.x = x.data_ptr()
    d.x_len = x.numel()
    d.y = y.data_ptr()
    return d


def dequantize_packed_batched(items, workspace=None, stream=None):
    """Decode many payloads in one launch.

    items: sequence of (fmt, shape, x_uint8_cuda, y_cuda) tuples.  The
    workspace (a CUDA uint8 tensor of ndq_batched_workspace_bytes(n) bytes)
    is allocated when not given; keep it alive until the stream passes.
    Returns the workspace tensor.
    """
    torch = _torch()
    descs = [make_desc(f, s, x, y) for (f, s, x, y) in items]
    nbytes = ndq_batched_workspace_bytes(len(descs))
    if workspace is None:
        dev = items[0][2].device if items else torch.device("cuda")
        workspace = torch.empty(max(16, nbytes), dtype=torch.uint8, device=dev)
    rc = ndq_dequantize_packed_batched(descs, workspace.data_ptr(), workspace.numel(), _stream_handle(stream))
    if rc:
        raise NdqError(rc)
    return workspace


def matmul_packed(fmt, w, N: int, K: int, x, out_dtype=None, y=None, stream=None, weight_dtype=None):
    """Y = X @ W^T with W [N, K] decoded from the CUDA uint8 payload `w`
    (binary32, or rounded to bfloat16 when weight_dtype is torch.bfloat16)
    and X a CUDA bfloat16 tensor [M, K]; returns Y [M, N]."""
    torch = _torch()
    out_dtype = out_dtype or torch.float32
    if x.dtype != torch.bfloat16 or not x.is_contiguous() or x.shape[-1] != K:
        raise ValueError("x must be a contiguous bfloat16 tensor [M, K]")
    M = x.numel() // K if K else x.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=out_dtype, device=w.device)
    wcode = out_dtype_code(weight_dtype or torch.float32)
    rc = ndq_matmul_packed(format_id(fmt), N, K, w.data_ptr(), w.numel(), x.data_ptr(), M, wcode,
                           out_dtype_code(y.dtype), y.data_ptr(), _stream_handle(stream))
    if rc:
        raise NdqError(rc, str(fmt))
    return y


def matmul_packed_batched(items, K: int, x, out_dtype=None, stream=None, weight_dtype=None):
    """Several products sharing the bfloat16 activations x [M, K]: items is
    a sequence of (fmt, w, N) or (fmt, w, N, y) with w a CUDA uint8 payload
    [N, K]; returns the list of outputs Y_i [M, N_i]."""
    torch = _torch()
    out_dtype = out_dtype or torch.float32
    if x.dtype != torch.bfloat16 or not x.is_contiguous() or x.shape[-1] != K:
        raise ValueError("x must be a contiguous bfloat16 tensor [M, K]")
    M = x.numel() // K if K else x.shape[0]
    descs, ys = [], []
    for it in items:
        fmt, w, N = it[0], it[1], it[2]
        y = it[3] if len(it) > 3 and it[3] is not None else torch.empty((M, N), dtype=out_dtype, device=w.device)
        descs.append(ndq_matmul_desc(format_id(fmt), 0, N, w.data_ptr(), w.numel(), y.data_ptr()))
        ys.append(y)
    wcode = out_dtype_code(weight_dtype or torch.float32)
    odt = out_dtype_code(ys[0].dtype if ys else out_dtype)
    rc = ndq_matmul_packed_batched(descs, K, x.data_ptr(), M, wcode, odt, _stream_handle(stream))
    if rc:
        raise NdqError(rc)
    return ys


def get_device_fault() -> int:
    return ndq_get_device_fault()


# ---- serving operators ------------------------------------------------------
# The tensor calls below launch on `stream` (a torch.cuda.Stream) or the current
# one.  What a call is given must be ready on that stream; outputs and
# workspaces that it is not given it makes on that stream.
def ndq_kv_plan(cached: int, fresh: int, n_req: int, block_size: int, free_blocks: int, free_count: int,
                block_table: int, table_width: int, q_start: int, kv_len: int, positions: int, slots: int,
                n_tokens: int, free_left: int, stream: int = 0) -> int:
    """Raw call (device pointers as integers); returns the status code."""
    return _lib.ndq_kv_plan(cached, fresh, n_req, block_size, free_blocks, free_count, block_table, table_width,
                            q_start, kv_len, positions, slots, n_tokens, free_left, stream)


def ndq_kv_append(cache, k: int, v: int, in_dtype: int, k_stride: int, v_stride: int, slots: int, n_tokens: int,
                  stream: int = 0) -> int:
    """Raw call; `cache` is an ndq_kv_cache; returns the status code."""
    return _lib.ndq_kv_append(cache, k, v, in_dtype, k_stride, v_stride, slots, n_tokens, stream)


def ndq_attention_workspace_bytes(head_dim: int) -> int:
    return _lib.ndq_attention_workspace_bytes(head_dim)


def ndq_attention_kv8(cache, q: int, dtype: int, n_tokens: int, q_heads: int, q_stride: int, block_table: int,
                      table_width: int, kv_len: int, q_start: int, n_req: int, max_q: int, scale: float, window: int,
                      out: int, lse: int, workspace: int, ws_bytes: int, stream: int = 0) -> int:
    """Raw call; `cache` is an ndq_kv_cache; returns the status code."""
    return _lib.ndq_attention_kv8(cache, q, dtype, n_tokens, q_heads, q_stride, block_table, table_width, kv_len,
                                  q_start, n_req, max_q, scale, window, out, lse, workspace, ws_bytes, stream)


def ndq_lora_workspace_bytes(M: int, max_rank: int, K: int) -> int:
    return _lib.ndq_lora_workspace_bytes(M, max_rank, K)


def ndq_lora_add(x: int, M: int, K: int, lora_a: int, lora_b: int, n_adapters: int, max_rank: int, N: int, ranks: int,
                 scales: int, index: int, base: int, dtype: int, y: int, workspace: int, ws_bytes: int,
                 stream: int = 0) -> int:
    """Raw call; returns the status code."""
    return _lib.ndq_lora_add(x, M, K, lora_a, lora_b, n_adapters, max_rank, N, ranks, scales, index, base, dtype, y,
                             workspace, ws_bytes, stream)


class _Torch:
    """What the wrappers of short launches look up in torch, once."""

    def __init__(self):
        torch = _torch()
        self.f32, self.bf16, self.i32, self.i64 = torch.float32, torch.bfloat16, torch.int32, torch.int64
        self.raw_stream = torch._C._cuda_getCurrentRawStream
        self.code = {torch.float32: NDQ_FLOAT, torch.float16: NDQ_FLOAT16, torch.bfloat16: NDQ_BFLOAT16}


_T = None


def _consts() -> _Torch:
    global _T
    _T = _Torch()
    return _T


def _raw_stream(stream, device: int) -> int:
    # (the handle alone: building a torch.cuda.Stream for each call costs microseconds)
    if stream is not None:
        return int(stream.cuda_stream)
    return (_T or _consts()).raw_stream(device)


def _same_device(what, device: int, *tensors):
    """Every tensor lies on GPU `device` (an index; -1, the host's, is none)."""
    for x in tensors:
        if x.get_device() != device or device < 0:
            raise ValueError(f"{what} takes CUDA tensors on one device")


def _made_for(stream, make):
    """make()'s tensors for a call on `stream` (None: the current one): from
    that stream's memory and filled in its order, so that what the call drops
    is not used by other streams while its kernels still run."""
    if stream is None:
        return make()
    with _torch().cuda.stream(stream):
        return make()


def _returned(stream, *tensors):
    """Tensors of _made_for that the caller gets, and may use and drop on the
    current stream."""
    if stream is not None:
        for x in tensors:
            x.record_stream(_torch().cuda.current_stream(x.device))


def _check(name, x, dtype, shape, device):
    if x.dtype != dtype or x.shape != shape or not x.is_contiguous() or x.device != device:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")


def _check_workspace(x, device: int):
    if x.get_device() != device or not x.is_contiguous():
        raise ValueError("the workspace must be contiguous, on the other tensors' device")


class KvCache:
    """An 8-bit key/value cache: codes k, v [blocks, kv_heads, block_size,
    head_dim] (torch.float8_e4m3fn or torch.int8) and binary32 scales k_scale,
    v_scale [blocks, kv_heads].  Keeps the tensors and their C descriptor."""

    def __init__(self, k, v, k_scale, v_scale):
        torch = _torch()
        code = {torch.float8_e4m3fn: NDQ_FLOAT8E4M3FN, torch.int8: NDQ_INT8}.get(k.dtype)
        if code is None or k.dim() != 4 or not k.is_cuda:
            raise ValueError("k must be a 4-D CUDA tensor of torch.float8_e4m3fn or torch.int8 codes")
        _check("k", k, k.dtype, k.shape, k.device)
        _check("v", v, k.dtype, k.shape, k.device)
        _check("k_scale", k_scale, torch.float32, k.shape[:2], k.device)
        _check("v_scale", v_scale, torch.float32, k.shape[:2], k.device)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.num_blocks, self.kv_heads, self.block_size, self.head_dim = k.shape
        self.device, self.gpu = k.device, k.get_device()
        self.desc = ndq_kv_cache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), self.num_blocks,
                                 self.kv_heads, self.block_size, self.head_dim, code)

    @classmethod
    def empty(cls, num_blocks: int, kv_heads: int, block_size: int, head_dim: int, dtype=None, device="cuda"):
        """A cache of uninitialised blocks (kv_append writes codes and scales)."""
        torch = _torch()
        shape = (num_blocks, kv_heads, block_size, head_dim)
        dtype = dtype or torch.float8_e4m3fn
        k, v = (torch.empty(shape, dtype=dtype, device=device) for _ in range(2))
        ks, vs = (torch.empty(shape[:2], dtype=torch.float32, device=device) for _ in range(2))
        return cls(k, v, ks, vs)


class KvPlan:
    """Output buffers of kv_plan: q_start [R + 1], kv_len [R], positions [T]
    (int32), slots [T] (int64), free_left [1] (int32).  Keeps the tensors and
    the arguments that name them to the library."""

    def __init__(self, q_start, kv_len, positions, slots, free_left):
        torch = _torch()
        R, T, device = kv_len.shape[0], slots.shape[0], kv_len.device
        self.gpu = kv_len.get_device()
        for name, x, dtype, n in (("q_start", q_start, torch.int32, R + 1), ("kv_len", kv_len, torch.int32, R),
                                  ("positions", positions, torch.int32, T), ("slots", slots, torch.int64, T),
                                  ("free_left", free_left, torch.int32, 1)):
            _check(name, x, dtype, (n,), device)
        self.q_start, self.kv_len, self.positions, self.slots, self.free_left = q_start, kv_len, positions, slots, free_left
        self.pointers = (q_start.data_ptr(), kv_len.data_ptr(), positions.data_ptr(), slots.data_ptr(), T, free_left.data_ptr())


def kv_plan_buffers(n_req: int, n_tokens: int, device="cuda") -> KvPlan:
    """Output buffers of kv_plan for n_req requests and up to n_tokens tokens."""
    torch = _torch()
    i32 = dict(dtype=torch.int32, device=device)
    return KvPlan(torch.empty(n_req + 1, **i32), torch.empty(n_req, **i32), torch.empty(n_tokens, **i32),
                  torch.empty(n_tokens, dtype=torch.int64, device=device), torch.empty(1, **i32))


def kv_plan(cached, fresh, block_size: int, free_blocks, free_count, block_table, out=None, n_tokens=None, stream=None):
    """Block tables and slot maps of one step (see ndq_kv_plan): cached, fresh
    [R], free_blocks [F], free_count [1] and block_table [R, width] are CUDA
    int32 tensors; block_table is written in place.  `out` holds the outputs,
    or `n_tokens` says how many tokens to allow for.  Returns the KvPlan.  Its
    kv_len and free_left may be the next step's cached and free_count, with
    other buffers for that step's outputs."""
    i32 = (_T or _consts()).i32
    if (cached.dtype is not i32 or fresh.dtype is not i32 or free_blocks.dtype is not i32 or free_count.dtype is not i32
            or block_table.dtype is not i32):
        raise ValueError("kv_plan takes int32 tensors")
    R, width = block_table.shape
    if cached.shape != (R,) or fresh.shape != (R,) or free_blocks.dim() != 1 or free_count.numel() != 1:
        raise ValueError("cached [R], fresh [R], block_table [R, width], free_blocks [F] and free_count [1] must agree")
    gpu = cached.get_device()
    _same_device("kv_plan", gpu, fresh, free_blocks, free_count, block_table)
    if not (cached.is_contiguous() and fresh.is_contiguous() and free_blocks.is_contiguous()
            and block_table.is_contiguous()):
        raise ValueError("kv_plan takes contiguous tensors")
    if out is None:
        if n_tokens is None:
            raise ValueError("kv_plan needs `out` or `n_tokens`")
        out = _made_for(stream, lambda: kv_plan_buffers(R, n_tokens, cached.device))
        _returned(stream, out.q_start, out.kv_len, out.positions, out.slots, out.free_left)
    elif out.kv_len.shape[0] != R or out.gpu != gpu:
        raise ValueError("out does not fit the requests")
    rc = _lib.ndq_kv_plan(cached.data_ptr(), fresh.data_ptr(), R, block_size, free_blocks.data_ptr(),
                          free_count.data_ptr(), block_table.data_ptr(), width, *out.pointers, _raw_stream(stream, gpu))
    if rc:
        raise NdqError(rc, "kv_plan")
    return out


def _row_stride(name, x, heads, dim):
    """Elements from one token's row [heads, dim] of x to the next."""
    shape = x.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim:
        raise ValueError(f"{name} must be [tokens, {heads}, {dim}]")
    st = x.stride()
    if st[2] != 1 or (st[1] != dim and heads > 1):
        raise ValueError(f"{name} must have dense heads")
    return st[0] if shape[0] > 1 else heads * dim


def kv_append(cache: KvCache, k, v, slots, stream=None) -> None:
    """Quantise the rows k, v [T, kv_heads, head_dim] (bfloat16 or float16;
    token strides of any multiple of 8) into `cache` at slots [T] (int64, as
    kv_plan writes them)."""
    c = _T or _consts()
    heads, dim, code = cache.kv_heads, cache.head_dim, c.code.get(k.dtype)
    T = k.shape[0] if k.dim() else -1
    if (k.dtype is not v.dtype or code is None or v.shape != k.shape or slots.dtype is not c.i64 or slots.shape != (T,)
            or not slots.is_contiguous()):
        raise ValueError("k and v must have the same type (bfloat16 or float16) and tokens, and slots one int64 for each")
    _same_device("kv_append", cache.gpu, k, v, slots)
    rc = _lib.ndq_kv_append(cache.desc, k.data_ptr(), v.data_ptr(), code, _row_stride("k", k, heads, dim),
                            _row_stride("v", v, heads, dim), slots.data_ptr(), T, _raw_stream(stream, cache.gpu))
    if rc:
        raise NdqError(rc, "kv_append")


def attention_workspace(n_req: int, n_tokens: int, q_heads: int, cache: KvCache, max_q: int = 1):
    """A workspace for attention_kv8 calls on `cache`, of any size: its
    counters are zeroed here, on the current stream, and left so by every
    call; calls that share it must not overlap.  (The sizes are accepted so
    that a caller need not know that they do not matter.)"""
    torch = _torch()
    ws = torch.empty(ndq_attention_workspace_bytes(cache.head_dim), dtype=torch.uint8, device=cache.device)
    ws[:4096].zero_()
    return ws


def attention_kv8(q, cache: KvCache, block_table, kv_len, q_start=None, max_q=None, scale=None, window: int = 0,
                  out=None, lse=None, workspace=None, stream=None):
    """Causal attention of q [T, q_heads, head_dim] (bfloat16 or float16) over
    `cache` (see ndq_attention_kv8): block_table [R, width], kv_len [R] and
    q_start [R + 1] are CUDA int32 tensors, q_start None when every request has
    one query.  max_q bounds the queries of one request (default: T, or 1).
    Returns out [T, q_heads, head_dim]; lse [T, q_heads] is written if given."""
    c = _T or _consts()
    i32, code = c.i32, c.code.get(q.dtype)
    if q.dim() != 3 or code is None:
        raise ValueError("q must be [tokens, q_heads, head_dim], bfloat16 or float16")
    T, H, D = q.shape
    qs = _row_stride("q", q, H, cache.head_dim)
    R, width = block_table.shape
    if (block_table.dtype is not i32 or kv_len.dtype is not i32 or kv_len.shape != (R,) or not block_table.is_contiguous()
            or not kv_len.is_contiguous()):
        raise ValueError("block_table must be int32 [R, width] and kv_len int32 [R]")
    gpu = cache.gpu
    _same_device("attention_kv8", gpu, q, block_table, kv_len)
    if q_start is not None and (q_start.dtype is not i32 or q_start.shape != (R + 1,) or not q_start.is_contiguous()
                                or q_start.get_device() != gpu):
        raise ValueError("q_start must be int32 [R + 1], on q's device")
    if out is None:
        out = _made_for(stream, lambda: _torch().empty((T, H, D), dtype=q.dtype, device=q.device))
        _returned(stream, out)
    elif out.dtype is not q.dtype or out.shape != q.shape or not out.is_contiguous() or out.get_device() != gpu:
        raise ValueError("out must be contiguous, of q's shape and type and on its device")
    if lse is not None and (lse.dtype is not c.f32 or lse.shape != (T, H) or not lse.is_contiguous() or lse.get_device() != gpu):
        raise ValueError("lse must be float32 [tokens, q_heads], on q's device")
    if workspace is not None:
        _check_workspace(workspace, gpu)
    else:
        workspace = _made_for(stream, lambda: attention_workspace(R, T, H, cache))
    rc = _lib.ndq_attention_kv8(
        cache.desc, q.data_ptr(), code, T, H, qs, block_table.data_ptr(), width, kv_len.data_ptr(),
        None if q_start is None else q_start.data_ptr(), R, max_q if max_q is not None else (1 if q_start is None else T),
        D ** -0.5 if scale is None else scale, window, out.data_ptr(), None if lse is None else lse.data_ptr(),
        workspace.data_ptr(), workspace.numel(), _raw_stream(stream, gpu))
    if rc:
        raise NdqError(rc, "attention_kv8")
    return out


def lora_workspace(M: int, n_adapters: int, max_rank: int, K: int, device="cuda"):
    """A workspace for lora_add calls of up to M rows, max_rank and K."""
    torch = _torch()
    return torch.empty(ndq_lora_workspace_bytes(M, max_rank, K), dtype=torch.uint8, device=device)


def lora_add(x, lora_a, lora_b, ranks, scales, index, base, out=None, workspace=None, stream=None):
    """base + scales[a] * (x A[a]^T) B[a]^T for each row's adapter a = index[m]
    (see ndq_lora_add): x bfloat16 [M, K], lora_a bfloat16 [n, rank, K], lora_b
    bfloat16 [n, N, rank], ranks int32 [n], scales float32 [n], index int32 [M],
    base float32 or bfloat16 [M, N].  out may be base.  Returns out."""
    c = _T or _consts()
    bf16, i32 = c.bf16, c.i32
    M, K = x.shape
    nA, rank, Ka = lora_a.shape
    nB, N, rb = lora_b.shape
    dtype = base.dtype
    if (x.dtype is not bf16 or lora_a.dtype is not bf16 or lora_b.dtype is not bf16 or Ka != K or nB != nA or rb != rank
            or base.shape != (M, N) or ranks.shape != (nA,) or scales.shape != (nA,) or index.shape != (M,) or ranks.dtype is not i32
            or index.dtype is not i32 or scales.dtype is not c.f32 or (dtype is not c.f32 and dtype is not bf16)):
        raise ValueError("lora_add: x [M, K], lora_a [n, r, K], lora_b [n, N, r] bfloat16, ranks [n], index [M] int32, "
                         "scales [n] float32, base [M, N] float32 or bfloat16")
    gpu = x.get_device()
    _same_device("lora_add", gpu, lora_a, lora_b, ranks, scales, index, base)
    if out is None:
        out = _made_for(stream, lambda: _torch().empty_like(base))
        _returned(stream, out)
    elif out.dtype is not dtype or out.shape != base.shape or out.get_device() != gpu:
        raise ValueError("out must have base's shape and type, on its device")
    if not (x.is_contiguous() and lora_a.is_contiguous() and lora_b.is_contiguous() and base.is_contiguous()
            and out.is_contiguous() and ranks.is_contiguous() and scales.is_contiguous() and index.is_contiguous()):
        raise ValueError("lora_add takes contiguous tensors")
    if workspace is not None:
        _check_workspace(workspace, gpu)
    else:
        workspace = _made_for(stream, lambda: lora_workspace(M, nA, rank, K, x.device))
    rc = _lib.ndq_lora_add(x.data_ptr(), M, K, lora_a.data_ptr(), lora_b.data_ptr(), nA, rank, N, ranks.data_ptr(),
                           scales.data_ptr(), index.data_ptr(), base.data_ptr(), c.code[dtype], out.data_ptr(),
                           workspace.data_ptr(), workspace.numel(), _raw_stream(stream, gpu))
    if rc:
        raise NdqError(rc, "lora_add")
    return out
