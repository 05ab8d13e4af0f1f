"""Python binding of the GB300 single-precision GEMM C library.

A thin ctypes layer over libsgemm_gb300.so (include/sgemm_gb300.h): the same
entry points under the same names, argument marshalling only.  Every step of
the computation runs in the library's CUDA kernels; there is no fallback, and
a missing library raises at the first call.  PyTorch, when used, supplies
device memory and the current stream (``gemm`` below), nothing else.
"""
from __future__ import annotations

import ctypes
import os
import threading

__all__ = [
    "SGEMM_OK", "SGEMM_ERR_CUDA", "SGEMM_ERR_TIMEOUT", "SGEMM_ERR_NOMEM",
    "SGEMM_ERR_UNSUPPORTED", "SGEMM_ERR_ARG", "SGEMM_ERR_SCRATCH", "PATH_AUTO", "PATH_FFMA",
    "PATH_3XTF32", "PATH_TF32", "PATH_GEMV", "ACT_NONE", "ACT_RELU", "sgemm_epilogue", "SgemmError", "library_path", "load",
    "sgemm", "sgemm_ex", "sgemm_host", "sgemm_plan", "sgemm_plan_detail", "sgemm_status_string",
    "sgemm_device_error", "sgemm_set_wait_limit", "sgemm_release_workspace",
    "sgemm_version", "sgemm_ffma_static_scratch", "sgemm_timing_enable",
    "sgemm_timing_read", "sgemm_launch_count", "sgemm_probe_tf32_rate", "gemm",
    "exported_symbols", "TYPE_F32", "TYPE_BF16", "TYPE_E4M3", "TYPE_E5M2",
    "sgemm_fp8_quantize", "fp8_quantize", "sgemm_fp8", "sgemm_fp8_plan", "fp8_gemm",
    "sgemm_moe", "moe", "ACT_SILU", "ACT_GELU", "sgemm_ffn", "ffn", "sgemm_ffn_backward",
    "ffn_backward", "sgemm_ffn_plan", "sgemm_q4_quantize", "q4_quantize", "sgemm_q4", "q4_gemm",
]

SGEMM_OK = 0
SGEMM_ERR_CUDA = 1
SGEMM_ERR_TIMEOUT = 2
SGEMM_ERR_NOMEM = 3
SGEMM_ERR_UNSUPPORTED = 4
SGEMM_ERR_ARG = 5
SGEMM_ERR_SCRATCH = 6

PATH_AUTO = 0
PATH_FFMA = 1
PATH_3XTF32 = 2
PATH_TF32 = 3
PATH_GEMV = 4
ACT_NONE = 0
ACT_RELU = 1
ACT_SILU = 2
ACT_GELU = 3

TYPE_F32 = 0
TYPE_BF16 = 1
TYPE_E4M3 = 2
TYPE_E5M2 = 3

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "libsgemm_gb300.so"
_lock = threading.Lock()
_lib = None


class SgemmError(RuntimeError):
    """A non-zero status returned by the library."""

    def __init__(self, status: int, where: str = "sgemm"):
        self.status = status
        super().__init__(f"{where}: status {status} ({sgemm_status_string(status)})")


class PlanInfo(ctypes.Structure):
    """sgemm_plan_info of the C header, field for field."""
    _fields_ = [(n, ctypes.c_int) for n in (
        "path", "tile_m", "tile_n", "vector", "ctas", "split", "dp_tiles", "pair", "fuse_a",
        "fuse_b", "wide", "accumulators", "k_block", "tail_nsplit", "sk_ctas", "sk_tail",
        "pre_transpose")]


def library_path() -> str:
    return os.path.join(_HERE, _LIB_NAME)


def _declare(lib):
    c, i64, f32, vp, i32 = ctypes.c_char, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_int
    gemm_args = [c, c, i64, i64, i64, f32, vp, i64, vp, i64, f32, vp, i64, vp]
    lib.sgemm.argtypes = gemm_args
    lib.sgemm.restype = i32
    lib.sgemm_ex.argtypes = gemm_args + [i32, i32]
    lib.sgemm_ex.restype = i32
    lib.sgemm_epilogue.argtypes = gemm_args[:13] + [vp, vp, i32, vp, i32, i32]
    lib.sgemm_epilogue.restype = i32
    lib.sgemm_host.argtypes = gemm_args
    lib.sgemm_host.restype = i32
    ip = ctypes.POINTER(ctypes.c_int)
    lib.sgemm_plan.argtypes = [c, c, i64, i64, i64, i64, i64, i64, i32, i32, i32, i32, i32, i32,
                               ip, ip, ip, ip, ip, ip]
    lib.sgemm_plan.restype = i32
    lib.sgemm_plan_detail.argtypes = [c, c, i64, i64, i64, i64, i64, i64, i32, i32, i32, i32, i32,
                                      i32, ctypes.POINTER(PlanInfo)]
    lib.sgemm_plan_detail.restype = i32
    lib.sgemm_status_string.argtypes = [i32]
    lib.sgemm_status_string.restype = ctypes.c_char_p
    lib.sgemm_device_error.argtypes = [vp]
    lib.sgemm_device_error.restype = i32
    lib.sgemm_set_wait_limit.argtypes = [ctypes.c_uint64]
    lib.sgemm_set_wait_limit.restype = i32
    lib.sgemm_release_workspace.argtypes = []
    lib.sgemm_release_workspace.restype = i32
    lib.sgemm_version.argtypes = []
    lib.sgemm_version.restype = i32
    lib.sgemm_timing_enable.argtypes = [i32]
    lib.sgemm_timing_enable.restype = i32
    lib.sgemm_timing_read.argtypes = [ctypes.POINTER(ctypes.c_float), i32]
    lib.sgemm_timing_read.restype = i32
    lib.sgemm_probe_tf32_rate.argtypes = [i32, ctypes.POINTER(ctypes.c_double)]
    lib.sgemm_probe_tf32_rate.restype = i32
    lib.sgemm_launch_count.argtypes = []
    lib.sgemm_launch_count.restype = i64
    lib.sgemm_ffma_static_scratch.argtypes = gemm_args + [i32]
    lib.sgemm_ffma_static_scratch.restype = i32
    lib.sgemm_fp8_quantize.argtypes = [i64, i64, vp, i32, i64, i32, i32, vp, i32, i64, vp, i64, vp]
    lib.sgemm_fp8_quantize.restype = i32
    lib.sgemm_fp8.argtypes = [c, c, i64, i64, i64, f32, vp, i32, i64, vp, i32, i64, vp, i32, i64, vp,
                              i32, i64, f32, vp, i32, i64, vp]
    lib.sgemm_fp8.restype = i32
    lib.sgemm_fp8_plan.argtypes = [i64, i64, i64, i32, i32, ip, ip, ip]
    lib.sgemm_fp8_plan.restype = i32
    lib.sgemm_moe.argtypes = [i64, i64, i64, i64, i64, vp, i32, i64, vp, vp, vp, vp, vp, vp, i64, i64,
                              vp, vp, i64, i64, i32, vp, i64, vp, vp, vp]
    lib.sgemm_moe.restype = i32
    lib.sgemm_ffn.argtypes = [i64, i64, i64, vp, i64, vp, vp, i64, vp, i64, i32, i32, vp, vp, i64, vp, vp, i64,
                              vp, i64, vp, i64, vp]
    lib.sgemm_ffn.restype = i32
    lib.sgemm_ffn_backward.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, vp, i64, vp, i64, i32, i32, vp, vp,
                                       i64, vp, vp, i64, vp, vp, vp, i64, vp, i64, i32, i32, vp, vp, i64, vp,
                                       i64, vp]
    lib.sgemm_ffn_backward.restype = i32
    lib.sgemm_ffn_plan.argtypes = [i64, i64, i64, i32, i32, ip, ip, ip]
    lib.sgemm_ffn_plan.restype = i32
    lib.sgemm_q4_quantize.argtypes = [i64, i64, vp, i32, i64, i32, vp, i64, vp, vp, i64, vp, i32, i64, vp]
    lib.sgemm_q4_quantize.restype = i32
    lib.sgemm_q4.argtypes = [i64, i64, i64, vp, i32, i64, vp, vp, vp, vp, vp, vp, i64, i64, i32, i32, vp, i32, i64, vp]
    lib.sgemm_q4.restype = i32


def load():
    """Loads the CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = library_path()
            if not os.path.exists(path):
                raise RuntimeError(
                    f"{path} is missing: build it with "
                    "`python -m dense_fp32_gemm_05_gb300.build` (needs nvcc)")
            lib = ctypes.CDLL(path)
            _declare(lib)
            _lib = lib
    return _lib


def exported_symbols(lib=None):
    """Names of the entry points this binding declares, for export checks."""
    return ["sgemm", "sgemm_ex", "sgemm_epilogue", "sgemm_host", "sgemm_plan", "sgemm_plan_detail",
            "sgemm_status_string", "sgemm_device_error",
            "sgemm_set_wait_limit", "sgemm_release_workspace", "sgemm_version",
            "sgemm_ffma_static_scratch", "sgemm_timing_enable", "sgemm_timing_read",
            "sgemm_launch_count", "sgemm_probe_tf32_rate", "sgemm_fp8_quantize",
            "sgemm_fp8", "sgemm_fp8_plan", "sgemm_moe", "sgemm_ffn", "sgemm_ffn_backward",
            "sgemm_ffn_plan", "sgemm_q4_quantize", "sgemm_q4"]


def _b(t: str) -> bytes:
    return t.encode() if isinstance(t, str) else bytes(t)


def _stream(stream) -> int | None:
    if stream is None:
        return None
    if isinstance(stream, int):
        return stream
    return int(getattr(stream, "cuda_stream", stream))


def sgemm(transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None) -> int:
    """C = alpha*op(A)*op(B) + beta*C; A, B, C are device addresses (int)."""
    return load().sgemm(_b(transA), _b(transB), M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
                        _stream(stream))


def sgemm_ex(transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None,
             path=PATH_AUTO, split=0) -> int:
    """sgemm with the path and the FFMA split-K factor forced."""
    return load().sgemm_ex(_b(transA), _b(transB), M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
                           _stream(stream), path, split)


def sgemm_epilogue(transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, row_scale=0,
                   bias=0, activation=ACT_NONE, stream=None, path=PATH_AUTO, split=0) -> int:
    """GEMM with the fused epilogue C = act(alpha * s_i * AB + beta * C + bias_j);
    row_scale / bias are device addresses (0 = none)."""
    return load().sgemm_epilogue(_b(transA), _b(transB), M, N, K, alpha, A, lda, B, ldb, beta,
                                 C, ldc, row_scale or None, bias or None, activation,
                                 _stream(stream), path, split)


def sgemm_host(transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None) -> int:
    """sgemm on HOST buffers (addresses as int), copies pipelined with the
    computation; asynchronous on `stream` (page-locked buffers overlap)."""
    return load().sgemm_host(_b(transA), _b(transB), M, N, K, alpha, A, lda, B, ldb, beta, C,
                             ldc, _stream(stream))


def sgemm_plan(transA, transB, M, N, K, lda, ldb, ldc, a_aligned=True, b_aligned=True,
               c_aligned=True, path=PATH_AUTO, split=0, num_sms=152):
    """The selector's decision, without a GPU: (status, dict)."""
    outs = [ctypes.c_int(0) for _ in range(6)]
    st = load().sgemm_plan(_b(transA), _b(transB), M, N, K, lda, ldb, ldc, int(a_aligned),
                           int(b_aligned), int(c_aligned), path, split, num_sms,
                           *[ctypes.byref(o) for o in outs])
    keys = ("path", "split", "tile_m", "tile_n", "vector", "ctas")
    return st, {k: o.value for k, o in zip(keys, outs)}


def sgemm_plan_detail(transA, transB, M, N, K, lda, ldb, ldc, a_aligned=True, b_aligned=True,
                      c_aligned=True, path=PATH_AUTO, split=0, num_sms=152):
    """The selector's decision down to the kernel variant, without a GPU:
    (status, dict of sgemm_plan_info's fields)."""
    info = PlanInfo()
    st = load().sgemm_plan_detail(_b(transA), _b(transB), M, N, K, lda, ldb, ldc, int(a_aligned),
                                  int(b_aligned), int(c_aligned), path, split, num_sms,
                                  ctypes.byref(info))
    return st, {name: getattr(info, name) for name, _ in PlanInfo._fields_}


def sgemm_status_string(status: int) -> str:
    return load().sgemm_status_string(status).decode()


def sgemm_device_error(stream=None) -> int:
    return load().sgemm_device_error(_stream(stream))


def sgemm_set_wait_limit(nanoseconds: int) -> int:
    return load().sgemm_set_wait_limit(nanoseconds)


def sgemm_release_workspace() -> int:
    return load().sgemm_release_workspace()


def sgemm_version() -> int:
    return load().sgemm_version()


def sgemm_timing_enable(n: int) -> int:
    """Record event pairs around the main kernel of the next n launches."""
    return load().sgemm_timing_enable(n)


def sgemm_probe_tf32_rate(reps: int = 4096):
    """Measured tcgen05 kind::tf32 rate: (status, multiply-adds per clock per SM)."""
    v = ctypes.c_double(0.0)
    st = load().sgemm_probe_tf32_rate(reps, ctypes.byref(v))
    return st, v.value


def sgemm_launch_count() -> int:
    """Kernels the library has launched in this process (all paths)."""
    return int(load().sgemm_launch_count())


def sgemm_timing_read(capacity: int = 4096):
    """Durations (ms) of the recorded main-kernel launches, oldest first."""
    buf = (ctypes.c_float * max(capacity, 1))()
    n = load().sgemm_timing_read(buf, capacity)
    if n < 0:
        raise SgemmError(-n, "sgemm_timing_read")
    return [float(buf[i]) for i in range(n)]


def sgemm_ffma_static_scratch(transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
                              stream=None, split=0) -> int:
    """The FFMA path with its split-K scratch in the library's static device
    array: allocates nothing (for callers that may not allocate device
    memory).  Overlapping calls on one device race on that array."""
    return load().sgemm_ffma_static_scratch(_b(transA), _b(transB), M, N, K, alpha, A, lda, B,
                                            ldb, beta, C, ldc, _stream(stream), split)


def gemm(A, B, C, transA="N", transB="N", alpha=1.0, beta=0.0, path=PATH_AUTO, split=0,
         stream=None):
    """Runs the library on torch CUDA tensors (marshalling only).

    A, B, C are 2-D float32 CUDA tensors holding the STORED row-major arrays
    (unit stride along the last dimension; stride(0) is the leading
    dimension).  C is updated in place.  Raises SgemmError on any non-zero
    status.  The call is asynchronous on ``stream`` (default: torch's current
    stream on C's device).
    """
    import torch  # local: only needed for this convenience wrapper

    for name, t in (("A", A), ("B", B), ("C", C)):
        if t.dtype != torch.float32 or not t.is_cuda or t.dim() != 2:
            raise ValueError(f"{name} must be a 2-D float32 CUDA tensor")
        if t.size(1) > 1 and t.stride(1) != 1:
            raise ValueError(f"{name} must have unit stride along its last dimension")
    M, N = C.shape
    K = A.shape[1] if transA.upper() == "N" else A.shape[0]
    if stream is None:
        stream = torch.cuda.current_stream(C.device)
    st = sgemm_ex(transA, transB, M, N, K, alpha, A.data_ptr(), max(A.stride(0), 1),
                  B.data_ptr(), max(B.stride(0), 1), beta, C.data_ptr(), max(C.stride(0), 1),
                  stream, path, split)
    if st != SGEMM_OK:
        raise SgemmError(st)
    return C


_types = {}
_TYPE_BYTES = -1                     # (no type of an operand: codes of 4 bits)


def _type_of(dtype):
    """The library's type code of a torch dtype (None: not one of its types)."""
    if not _types:
        import torch
        _types.update({torch.float32: TYPE_F32, torch.bfloat16: TYPE_BF16,
                       torch.float8_e4m3fn: TYPE_E4M3, torch.float8_e5m2: TYPE_E5M2,
                       torch.uint8: _TYPE_BYTES})
    return _types.get(dtype)


_FLOATS, _CODES, _SCALES = (TYPE_F32, TYPE_BF16), (TYPE_E4M3, TYPE_E5M2), (TYPE_F32,)


def _matrix(name, t, types, device=None):
    """(address, type, leading dimension, rows, columns) of a 2-D row-major CUDA
    tensor on `device` (an index).  Rows may not overlap: one that is broadcast over
    others (stride 0) is refused.  Small calls take as long as this takes."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    rows, cols = t.shape
    ld, unit = t.stride()
    code = _types.get(t.dtype) if _types else _type_of(t.dtype)
    if code not in types or not t.is_cuda or (unit != 1 and cols > 1):
        raise ValueError(f"{name} must be a 2-D CUDA tensor of a type the call takes, with unit "
                         "stride along its last dimension")
    if device is not None and t.get_device() != device:
        raise ValueError("the operands must be on one device")
    if rows <= 1:
        ld = cols                    # (a single row's stride means nothing)
    elif ld < cols:
        raise ValueError(f"{name}'s rows overlap (strides {(ld, unit)}, {cols} columns): give it "
                         "contiguous")
    return t.data_ptr(), code, ld or 1, rows, cols


_raw_stream = None


def _current_stream(device):
    """torch's current stream on a device (an index) as an address."""
    global _raw_stream
    if _raw_stream is None:
        import torch
        # (the public current_stream() builds an object: 2 us on a Grace core)
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda index: torch.cuda.current_stream(index).cuda_stream)
    return _raw_stream(device)


_raw_device = None


def _check_device(device):
    """The library launches on the current device: tensors of another are refused."""
    global _raw_device
    if _raw_device is None:
        import torch
        _raw_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    if _raw_device() != device:
        raise ValueError(f"the operands are on device {device}, which is not the current one")


def _new(shape, dtype, device, stream, ld=None):
    """A tensor for a call's result: of the stream that the call runs on, so that torch gives
    it no memory that work on another stream still uses.  ld: a matrix' row stride."""
    import torch
    if stream is not None:
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(_stream(stream), device=device)
        with torch.cuda.stream(stream):
            return _new(shape, dtype, device, None, ld)
    if ld is None or ld == shape[1]:
        return torch.empty(shape, device=device, dtype=dtype)
    # (an empty tensor's columns taken off cost 2 us more)
    return torch.empty_strided(shape, (ld, 1), device=device, dtype=dtype)


def sgemm_fp8_quantize(rows, cols, X, x_type, ldx, group_rows, group_cols, Q, q_type, ldq, S, lds,
                       stream=None) -> int:
    """Codes Q and scales S of the rows x cols matrix X; device addresses (int)."""
    return load().sgemm_fp8_quantize(rows, cols, X, x_type, ldx, group_rows, group_cols, Q, q_type,
                                     ldq, S, lds, _stream(stream))


def fp8_quantize(X, group=(1, 128), dtype=None, Q=None, S=None, stream=None):
    """(codes, scales) of a 2-D float32 or bfloat16 CUDA tensor, with one scale for
    each group of 1 x 128, 128 x 1 or 128 x 128 values.

    Codes are of ``dtype`` (torch.float8_e4m3fn by default, or float8_e5m2);
    scales are float32, of shape (ceil(cols / 128), rows), (ceil(rows / 128),
    cols) or (ceil(rows / 128), ceil(cols / 128)).  ``Q`` and ``S`` take
    buffers to write into; new ones belong to the stream of the call.  The tensors
    are on the current device.  Asynchronous on ``stream`` (default: torch's current
    stream); raises SgemmError on any non-zero status.
    """
    device = X.get_device()
    px, tx, ldx, rows, cols = _matrix("X", X, _FLOATS)
    _check_device(device)
    gr, gc = group
    if Q is None:
        import torch
        Q = _new((rows, cols), dtype or torch.float8_e4m3fn, X.device, stream)
    elif dtype is not None and dtype != Q.dtype:
        raise ValueError("Q is not of the given dtype")
    pq, tq, ldq, q_rows, q_cols = _matrix("Q", Q, _CODES, device)
    s_rows, s_cols = (((cols + 127) // 128, rows) if gr == 1 else
                      ((rows + 127) // 128, cols if gc == 1 else (cols + 127) // 128))
    if S is None:
        import torch
        S = _new((s_rows, s_cols), torch.float32, X.device, stream)
    ps, _, lds, have_rows, have_cols = _matrix("S", S, _SCALES, device)
    if q_rows != rows or q_cols != cols or have_rows != s_rows or have_cols != s_cols:
        raise ValueError(f"Q must have X's shape and S the shape ({s_rows}, {s_cols})")
    st = load().sgemm_fp8_quantize(rows, cols, px, tx, ldx, gr, gc, pq, tq, ldq, ps, lds,
                                   _current_stream(device) if stream is None else _stream(stream))
    if st != SGEMM_OK:
        raise SgemmError(st, "sgemm_fp8_quantize")
    return Q, S


def sgemm_fp8(transA, transB, M, N, K, alpha, A, a_type, lda, SA, a_group, ldsa, B, b_type, ldb, SB,
              b_group, ldsb, beta, C, c_type, ldc, stream=None) -> int:
    """C = alpha*op(A)*op(B) + beta*C with quantised A and B; device addresses (int)."""
    return load().sgemm_fp8(_b(transA), _b(transB), M, N, K, alpha, A, a_type, lda, SA, a_group, ldsa,
                            B, b_type, ldb, SB, b_group, ldsb, beta, C, c_type, ldc, _stream(stream))


def sgemm_fp8_plan(M, N, K, b_group=128, num_sms=152):
    """The 8-bit product's tile and cluster size, without a GPU: (status, dict)."""
    outs = [ctypes.c_int(0) for _ in range(3)]
    st = load().sgemm_fp8_plan(M, N, K, b_group, num_sms, *[ctypes.byref(o) for o in outs])
    return st, {k: o.value for k, o in zip(("tile_m", "tile_n", "ksplit"), outs)}


def fp8_gemm(A, SA, B, SB, C, transA="N", transB="T", alpha=1.0, beta=0.0, a_group=1, b_group=128,
             stream=None):
    """C = alpha*op(A)*op(B) + beta*C of quantised operands; C is updated in place and returned.

    A and B are 2-D CUDA tensors of codes (float8_e4m3fn or float8_e5m2) holding the
    STORED arrays, SA and SB their float32 scales as ``fp8_quantize`` lays them
    out; C is float32 or bfloat16.  ``a_group`` 1: A has a scale for each row of
    op(A) and 128 of the sum (groups of 1 x 128 for transA 'N', 128 x 1 for 'T');
    128: for each 128 x 128 block.  ``b_group`` likewise.  A linear layer's forward
    product is the default layout, x (1 x 128) times W^T (128 x 128 blocks).
    The tensors are on the current device.  Asynchronous on ``stream`` (default:
    torch's current stream); raises SgemmError on any non-zero status.
    """
    device = C.get_device()
    pa, a_type, lda, a_rows, a_cols = _matrix("A", A, _CODES, device)
    pb, b_type, ldb, b_rows, b_cols = _matrix("B", B, _CODES, device)
    pc, c_type, ldc, M, N = _matrix("C", C, _FLOATS)
    _check_device(device)
    psa, _, ldsa, sa_rows, sa_cols = _matrix("SA", SA, _SCALES, device)
    psb, _, ldsb, sb_rows, sb_cols = _matrix("SB", SB, _SCALES, device)
    a_trans, b_trans = transA in "TtCc", transB in "TtCc"
    K, a_m = (a_rows, a_cols) if a_trans else (a_cols, a_rows)
    b_n, b_k = (b_rows, b_cols) if b_trans else (b_cols, b_rows)
    if a_m != M or b_n != N or b_k != K:
        raise ValueError("the shapes of A, B and C do not fit together")
    kb = (K + 127) // 128
    if ((sa_rows != kb or sa_cols != M) if a_group == 1 else
            (sa_rows != (a_rows + 127) // 128 or sa_cols != (a_cols + 127) // 128)):
        raise ValueError("SA's shape does not fit A and its groups")
    if ((sb_rows != kb or sb_cols != N) if b_group == 1 else
            (sb_rows != (b_rows + 127) // 128 or sb_cols != (b_cols + 127) // 128)):
        raise ValueError("SB's shape does not fit B and its groups")
    st = load().sgemm_fp8(_b(transA), _b(transB), M, N, K, alpha, pa, a_type, lda, psa, a_group, ldsa,
                          pb, b_type, ldb, psb, b_group, ldsb, beta, pc, c_type, ldc,
                          _current_stream(device) if stream is None else _stream(stream))
    if st != SGEMM_OK:
        raise SgemmError(st, "sgemm_fp8")
    return C


def sgemm_moe(T, D, F, E, topk, x, x_type, ldx, router, logits, gate, s_gate, up, s_up, ld_in,
              stride_in, down, s_down, ld_down, stride_down, renormalize, y, ldy, indices, weights,
              stream=None) -> int:
    """A mixture-of-experts layer for a few tokens; device addresses (int), router 0 = none."""
    return load().sgemm_moe(T, D, F, E, topk, x, x_type, ldx, router or None, logits, gate, s_gate, up,
                            s_up, ld_in, stride_in, down, s_down, ld_down, stride_down,
                            int(renormalize), y, ldy, indices, weights, _stream(stream))


def _experts(name, t, shape, device):
    """(address, row stride, matrix stride) of matrices of E4M3 codes."""
    if t.shape != shape or _type_of(t.dtype) != TYPE_E4M3 or t.get_device() != device:
        raise ValueError(f"{name} must be a CUDA tensor of float8_e4m3fn codes of shape {shape} "
                         "on the operands' device")
    stride, ld, unit = t.stride()
    if unit != 1:
        raise ValueError(f"{name} must have unit stride along its last dimension")
    return t.data_ptr(), ld, stride


def _packed(name, t, shape, dtype, device):
    if t.shape != shape or t.dtype != dtype or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor of shape {shape} on the "
                         "operands' device")
    return t.data_ptr()


def moe(x, router, gate, s_gate, up, s_up, down, s_down, topk, renormalize=True, y=None, logits=None,
        indices=None, weights=None, stream=None):
    """(y, logits, indices, weights): a mixture-of-experts layer for up to 128 tokens.

    x: T x D, float32 or bfloat16.  router: E x D float32, or None with ``logits``
    (T x E float32) given.  gate and up: E x F x D codes (float8_e4m3fn) with
    128 x 128 block scales s_gate, s_up (E x ceil(F/128) x ceil(D/128)); down:
    E x D x F with s_down; rows of codes start on 16 bytes (pad them where D or F
    is no multiple of 16).  Each token takes its ``topk`` experts of the largest
    logits with their softmax weights (``renormalize``: divided by their sum);
    an expert is down (silu(gate x) * (up x)).  y, logits, indices (int32) and
    weights take buffers to write into; new ones belong to the stream of the call.
    The tensors are on the current device.  Asynchronous on ``stream`` (default:
    torch's current stream); raises SgemmError on any non-zero status.
    """
    import torch

    f32, i32 = torch.float32, torch.int32
    device = x.get_device()
    px, x_type, ldx, T, D = _matrix("x", x, _FLOATS)
    _check_device(device)
    E, F, _ = gate.shape
    inner, outer = (E, F, D), (E, D, F)
    pg, ld_in, stride_in = _experts("gate", gate, inner, device)
    pu, ld_up, stride_up = _experts("up", up, inner, device)
    pd, ld_down, stride_down = _experts("down", down, outer, device)
    if ld_up != ld_in or stride_up != stride_in:
        raise ValueError("gate and up must have the same strides")
    fb, db = (F + 127) // 128, (D + 127) // 128
    in_blocks, out_blocks, chosen = (E, fb, db), (E, db, fb), (T, topk)
    if router is None and logits is None:
        raise ValueError("give router or logits")
    if logits is None:
        logits = _new((T, E), f32, x.device, stream)
    if y is None:
        y = _rows_on_16(T, D, x, stream)
    if indices is None:
        indices = _new(chosen, i32, x.device, stream)
    if weights is None:
        weights = _new(chosen, f32, x.device, stream)
    py, y_type, ldy, y_rows, y_cols = _matrix("y", y, _FLOATS, device)
    if y_type != x_type or y_rows != T or y_cols != D:
        raise ValueError("y must have x's shape and dtype")
    st = load().sgemm_moe(
        T, D, F, E, topk, px, x_type, ldx,
        None if router is None else _packed("router", router, (E, D), f32, device),
        _packed("logits", logits, (T, E), f32, device), pg, _packed("s_gate", s_gate, in_blocks, f32, device),
        pu, _packed("s_up", s_up, in_blocks, f32, device), ld_in, stride_in,
        pd, _packed("s_down", s_down, out_blocks, f32, device), ld_down, stride_down, int(renormalize), py,
        ldy, _packed("indices", indices, chosen, i32, device), _packed("weights", weights, chosen, f32, device),
        _current_stream(device) if stream is None else _stream(stream))
    if st != SGEMM_OK:
        raise SgemmError(st, "sgemm_moe")
    return y, logits, indices, weights


def sgemm_ffn(T, D, F, x, ldx, gate, up, ld_in, down, ld_down, activation, kept_type, g, u, ld_kept, sg, su,
              ld_scales, h, ldh, y, ldy, stream=None) -> int:
    """A gated feed-forward block's forward pass; device addresses (int), 0 = none."""
    return load().sgemm_ffn(T, D, F, x, ldx, gate, up, ld_in, down, ld_down, activation, kept_type, g or None,
                            u or None, ld_kept, sg or None, su or None, ld_scales, h, ldh, y, ldy,
                            _stream(stream))


def sgemm_ffn_backward(T, D, F, dy, lddy, x, ldx, gate, up, ld_in, down, ld_down, activation, kept_type, g, u,
                       ld_kept, sg, su, ld_scales, dg, du, h, ldh, dx, lddx, grad_type, accumulate, dgate, dup,
                       ld_din, ddown, ld_ddown, stream=None) -> int:
    """A gated feed-forward block's gradients; device addresses (int)."""
    return load().sgemm_ffn_backward(T, D, F, dy, lddy, x, ldx, gate, up, ld_in, down, ld_down, activation,
                                     kept_type, g, u, ld_kept, sg or None, su or None, ld_scales, dg, du, h, ldh,
                                     dx, lddx, grad_type, int(accumulate), dgate, dup, ld_din, ddown, ld_ddown,
                                     _stream(stream))


def sgemm_ffn_plan(T, D, F, kept_type=TYPE_BF16, num_sms=152):
    """How a block's launches are cut, without a GPU: (status, dict of (rows, columns, split))."""
    rows, cols, split = ((ctypes.c_int * 5)() for _ in range(3))
    st = load().sgemm_ffn_plan(T, D, F, kept_type, num_sms, rows, cols, split)
    return st, {k: (rows[i], cols[i], split[i]) for i, k in enumerate(("gated", "down", "slope", "dx", "weights"))}


_BF16, _KEPT = (TYPE_BF16,), (TYPE_BF16, TYPE_E4M3)


def _of_shape(name, t, types, shape, device):
    """(address, type, leading dimension) of a matrix of a given shape, on `device`."""
    if t.shape == shape and t.get_device() == device:    # (0.3 us less than what _matrix looks at)
        rows, cols = shape
        ld, unit = t.stride()
        code = _types.get(t.dtype)
        if code in types and (unit == 1 or cols <= 1) and (ld >= cols or rows <= 1):
            return t.data_ptr(), code, (ld if rows > 1 else cols) or 1
    p, code, ld, rows, cols = _matrix(name, t, types, device)
    if (rows, cols) != shape:
        raise ValueError(f"{name} must have the shape {shape}")
    return p, code, ld


def _ffn_weights(x, gate, up, down):
    """The checked arguments that both passes begin with."""
    device = x.get_device()
    px, _, ldx, T, D = _matrix("x", x, _BF16)
    _check_device(device)
    F = gate.shape[0] if gate.dim() == 2 else -1
    shape = (F, D)
    pg, _, ld_in = _of_shape("gate", gate, _BF16, shape, device)
    pu, _, ld_up = _of_shape("up", up, _BF16, shape, device)
    if ld_in != ld_up:
        raise ValueError("gate and up must have the same strides")
    pd, _, ld_down = _of_shape("down", down, _BF16, (D, F), device)
    return device, T, D, F, px, ldx, pg, pu, ld_in, pd, ld_down


def _ffn_kept(kept, T, F, device):
    """(type, g, u, leading dimension, sg, su, leading dimension of the scales)."""
    if len(kept) not in (2, 4):
        raise ValueError("kept holds g and u, and with 8-bit codes their scales")
    shape = (T, F)
    pg, code, ld = _of_shape("kept g", kept[0], _KEPT, shape, device)
    pu, code_u, ld_u = _of_shape("kept u", kept[1], _KEPT, shape, device)
    if ld != ld_u:
        raise ValueError("kept g and u must have the same strides")
    if code != code_u or (code == TYPE_E4M3) != (len(kept) == 4):
        raise ValueError("kept holds g and u in bfloat16, or in float8_e4m3fn and their scales")
    if len(kept) == 2:
        return code, pg, pu, ld, None, None, 1
    shape = ((F + 127) // 128, T)
    psg, _, lds = _of_shape("scales of g", kept[2], _BF16, shape, device)
    psu, _, lds_u = _of_shape("scales of u", kept[3], _BF16, shape, device)
    if lds != lds_u:
        raise ValueError("the scales must have the same strides")
    # (one row of scales, whose stride means nothing, still has a token in each column)
    return code, pg, pu, ld, psg, psu, lds


def _scratch_rows(T, F, like, stream):
    """A T x F bf16 matrix whose rows start on 128 bytes: TMA reads them in whole lines
    (gradients of 777 x 1000 x 2501 32.7 us, with rows on 16 bytes 40.9)."""
    return _new((T, F), like.dtype, like.device, stream, (F + 63) // 64 * 64)


def _rows_on_16(T, D, like, stream):
    """A T x D bf16 matrix whose rows start on 16 bytes, so that it may be another block's x or dy."""
    return _new((T, D), like.dtype, like.device, stream, (D + 7) // 8 * 8)


def ffn(x, gate, up, down, activation=ACT_SILU, keep=None, kept=None, y=None, h=None, stream=None):
    """(y, kept): a gated feed-forward block, y = (act(x gate^T) * (x up^T)) down^T.

    x: T x D, gate and up: F x D (with the same strides), down: D x F, all bfloat16 CUDA
    tensors whose rows start on 16 bytes (pad them where D or F is no multiple of 8).
    ``activation``: ACT_SILU, ACT_GELU (tanh form), ACT_RELU or ACT_NONE.  ``keep``:
    torch.bfloat16 or torch.float8_e4m3fn keeps x gate^T and x up^T for
    ``ffn_backward`` as (g, u), or as (g, u, sg, su): codes, and bfloat16 scales
    of shape (ceil(F / 128), T) for each 128 columns of a row; None keeps nothing,
    and kept is None.  ``kept``, ``y`` and ``h`` (T x F, the product's other operand, rows on
    16 bytes) take buffers to write into; new ones belong to the stream of the call, and
    have rows that start on 16 bytes, as the next block's x does (y's are padded where D is no
    multiple of 8).  The tensors are on the current device.  Asynchronous on ``stream`` (default:
    torch's current stream); raises SgemmError on any non-zero status.
    """
    device, T, D, F, px, ldx, pg, pu, ld_in, pd, ld_down = _ffn_weights(x, gate, up, down)
    if kept is None and keep is not None:
        import torch
        if keep not in (torch.bfloat16, torch.float8_e4m3fn):
            raise ValueError("keep must be torch.bfloat16, torch.float8_e4m3fn or None")
        kept = tuple(_new((T, F), keep, x.device, stream, (F + 15) // 16 * 16) for _ in range(2))
        if keep != torch.bfloat16:
            kept += tuple(_new(((F + 127) // 128, T), torch.bfloat16, x.device, stream) for _ in range(2))
    elif kept is not None and keep is not None and kept[0].dtype != keep:
        raise ValueError("kept is not of the type that keep asks for")
    k = (TYPE_BF16, None, None, max(F, 1), None, None, 1) if kept is None else _ffn_kept(kept, T, F, device)
    if y is None:
        y = _rows_on_16(T, D, x, stream)
    if h is None:
        h = _scratch_rows(T, F, x, stream)
    py, _, ldy = _of_shape("y", y, _BF16, (T, D), device)
    ph, _, ldh = _of_shape("h", h, _BF16, (T, F), device)
    st = load().sgemm_ffn(T, D, F, px, ldx, pg, pu, ld_in, pd, ld_down, activation, *k, ph, ldh, py, ldy,
                          _current_stream(device) if stream is None else _stream(stream))
    if st != SGEMM_OK:
        raise SgemmError(st, "sgemm_ffn")
    return y, kept


def ffn_backward(dy, x, gate, up, down, kept, activation=ACT_SILU, dx=None, dgate=None, dup=None, ddown=None,
                 accumulate=False, scratch=None, stream=None):
    """(dx, dgate, dup, ddown): the gradients of ``ffn``'s x, gate, up and down.

    dy: T x D bfloat16, rows on 16 bytes like x; ``kept`` and ``activation`` as ``ffn`` had
    them.  dx is bfloat16; dgate, dup and ddown are bfloat16 or, in buffers given,
    all float32.  ``accumulate`` adds to the three weight gradients (which are given
    then).  ``scratch``: three T x F bfloat16 buffers with the same strides, rows on
    16 bytes (on 128, as new ones have them, they are read faster).  New weight gradients are
    contiguous; a new dx has rows on 16 bytes, as the block before takes its dy.
    Buffers, device, stream and errors as in ``ffn``.
    """
    device, T, D, F, px, ldx, pg, pu, ld_in, pd, ld_down = _ffn_weights(x, gate, up, down)
    pdy, _, lddy = _of_shape("dy", dy, _BF16, (T, D), device)
    k = _ffn_kept(kept, T, F, device)
    if accumulate and (dgate is None or dup is None or ddown is None):
        raise ValueError("accumulate needs the three weight gradients")
    if dx is None:
        dx = _rows_on_16(T, D, x, stream)
    if dgate is None:
        dgate = _new((F, D), x.dtype, x.device, stream)
    if dup is None:
        dup = _new((F, D), x.dtype, x.device, stream)
    if ddown is None:
        ddown = _new((D, F), x.dtype, x.device, stream)
    if scratch is None:
        scratch = tuple(_scratch_rows(T, F, x, stream) for _ in range(3))
    if len(scratch) != 3:
        raise ValueError("scratch is three buffers")
    shape = (T, F)
    p0, _, ld0 = _of_shape("scratch 0", scratch[0], _BF16, shape, device)
    p1, _, ld1 = _of_shape("scratch 1", scratch[1], _BF16, shape, device)
    p2, _, ld2 = _of_shape("scratch 2", scratch[2], _BF16, shape, device)
    if ld0 != ld1 or ld0 != ld2:
        raise ValueError("the scratch buffers must have the same strides")
    pdx, _, lddx = _of_shape("dx", dx, _BF16, (T, D), device)
    shape = (F, D)
    pdg, grad, ld_din = _of_shape("dgate", dgate, _FLOATS, shape, device)
    pdu, grad_up, ld_dup = _of_shape("dup", dup, _FLOATS, shape, device)
    if ld_din != ld_dup:
        raise ValueError("dgate and dup must have the same strides")
    pdd, grad_down, ld_ddown = _of_shape("ddown", ddown, _FLOATS, (D, F), device)
    if grad != grad_up or grad != grad_down:
        raise ValueError("the weight gradients must be of one type")
    st = load().sgemm_ffn_backward(
        T, D, F, pdy, lddy, px, ldx, pg, pu, ld_in, pd, ld_down, activation, *k, p0, p1, p2, ld0,
        pdx, lddx, grad, 1 if accumulate else 0, pdg, pdu, ld_din, pdd, ld_ddown,
        _current_stream(device) if stream is None else _stream(stream))
    if st != SGEMM_OK:
        raise SgemmError(st, "sgemm_ffn_backward")
    return dx, dgate, dup, ddown


def sgemm_q4_quantize(rows, cols, X, x_type, ldx, group, Q, ldq, S, Z, lds, V=0, v_type=TYPE_F32, ldv=1,
                      stream=None) -> int:
    """4-bit codes Q, scales S and zero codes Z of X; device addresses (int), Z or V 0 = none."""
    return load().sgemm_q4_quantize(rows, cols, X, x_type, ldx, group, Q, ldq, S, Z or None, lds, V or None,
                                    v_type, ldv, _stream(stream))


def sgemm_q4(M, N, K, X, x_type, ldx, Q, S, Z, Q2, S2, Z2, ldq, lds, group, activation, C, c_type, ldc,
             stream=None) -> int:
    """C = X W^T or act(X W^T) * (X W2^T) with 4-bit matrices; device addresses (int), 0 = none."""
    return load().sgemm_q4(M, N, K, X, x_type, ldx, Q, S, Z or None, Q2 or None, S2 or None, Z2 or None, ldq, lds,
                           group, activation, C, c_type, ldc, _stream(stream))


def _bytes(name, t, shape, device):
    """(address, row stride) of a matrix of bytes."""
    if t.shape != shape or _type_of(t.dtype) != _TYPE_BYTES or t.get_device() != device:
        raise ValueError(f"{name} must be a CUDA tensor of uint8 of shape {shape} on the operands' device")
    ld, unit = t.stride()
    if (unit != 1 and shape[1] > 1) or (ld < shape[1] and shape[0] > 1):
        raise ValueError(f"{name} must have unit stride along its last dimension and rows that do not overlap")
    return t.data_ptr(), (ld if shape[0] > 1 else shape[1]) or 1


def q4_quantize(W, group=128, symmetric=True, Q=None, S=None, Z=None, V=None, stream=None):
    """(codes, scales, zero codes) of a 2-D float32 or bfloat16 CUDA tensor, 4 bits each.

    Codes are uint8 of shape (rows, ceil(cols / 2)), the even column in a byte's low half;
    new ones have rows that start on 16 bytes, as ``q4_gemm`` reads them.  Scales are
    float32 and zero codes uint8 of shape (ceil(cols / group), rows), for groups of 32, 64 or 128 in a
    row; ``symmetric``: no zero codes, and the result's third is None.  ``Q``, ``S``, ``Z`` take
    buffers to write into; new ones belong to the stream of the call.  ``V`` (W's shape,
    float32 or bfloat16) takes the codes' values.  The tensors are on the current device.
    Asynchronous on ``stream`` (default: torch's current stream); raises SgemmError on any
    non-zero status.
    """
    device = W.get_device()
    pw, w_type, ldw, rows, cols = _matrix("W", W, _FLOATS)
    _check_device(device)
    if group not in (32, 64, 128):
        raise ValueError("group must be 32, 64 or 128")
    if symmetric and Z is not None:
        raise ValueError("symmetric codes have no zero codes")
    half, groups = (cols + 1) // 2, (cols + group - 1) // group
    if Q is None or S is None or Z is None and not symmetric:
        import torch
    if Q is None:
        Q = _new((rows, half), torch.uint8, W.device, stream, (half + 15) // 16 * 16)
    if S is None:
        S = _new((groups, rows), torch.float32, W.device, stream)
    if Z is None and not symmetric:
        Z = _new((groups, rows), torch.uint8, W.device, stream)
    pq, ldq = _bytes("Q", Q, (rows, half), device)
    ps, _, lds = _of_shape("S", S, _SCALES, (groups, rows), device)
    pz = None
    if Z is not None:
        pz, ldz = _bytes("Z", Z, (groups, rows), device)
        if ldz != lds:
            raise ValueError("S and Z must have the same strides")
    pv, v_type, ldv = (None, TYPE_F32, 1) if V is None else _of_shape("V", V, _FLOATS, (rows, cols), device)
    st = load().sgemm_q4_quantize(rows, cols, pw, w_type, ldw, group, pq, ldq, ps, pz, lds, pv, v_type, ldv,
                                  _current_stream(device) if stream is None else _stream(stream))
    if st != SGEMM_OK:
        raise SgemmError(st, "sgemm_q4_quantize")
    return Q, S, Z


def q4_gemm(X, Q, S, C=None, Z=None, Q2=None, S2=None, Z2=None, group=128, activation=None, dtype=None,
            stream=None):
    """X W^T, or act(X W^T) * (X W2^T), for a few rows of X and 4-bit matrices.

    X: M x K, bfloat16 or float32.  Q, S, Z (and Q2, S2, Z2 with the same strides): codes,
    scales and zero codes (None: symmetric) of N x K matrices as ``q4_quantize`` makes them
    with that ``group``; rows of codes start on 16 bytes.  ``activation``: of two matrices,
    ACT_SILU by default.  C: M x N, bfloat16 or float32, written and returned; a new one is
    of ``dtype`` (default X's) and belongs to the stream of the call.  The weights are
    read once for each 64 rows of X (32 in float32).  The tensors are on the current
    device.  Asynchronous on ``stream`` (default: torch's current stream); raises
    SgemmError on any non-zero status.
    """
    device = X.get_device()
    px, x_type, ldx, M, K = _matrix("X", X, _FLOATS)
    _check_device(device)
    if group not in (32, 64, 128):
        raise ValueError("group must be 32, 64 or 128")
    N = Q.shape[0]
    codes, scales = (N, (K + 1) // 2), ((K + group - 1) // group, N)
    pq, ldq = _bytes("Q", Q, codes, device)
    ps, _, lds = _of_shape("S", S, _SCALES, scales, device)
    pz = p2 = ps2 = pz2 = None
    if Z is not None:
        pz, ldz = _bytes("Z", Z, scales, device)
        if ldz != lds:
            raise ValueError("S and Z must have the same strides")
    if Q2 is not None:
        p2, ldq2 = _bytes("Q2", Q2, codes, device)
        ps2, _, lds2 = _of_shape("S2", S2, _SCALES, scales, device)
        if (Z2 is None) != (Z is None):
            raise ValueError("Z and Z2 are both given or neither")
        ldz2 = lds
        if Z2 is not None:
            pz2, ldz2 = _bytes("Z2", Z2, scales, device)
        if ldq2 != ldq or lds2 != lds or ldz2 != lds:
            raise ValueError("both matrices must have the same strides")
    elif S2 is not None or Z2 is not None:
        raise ValueError("S2 and Z2 belong to Q2")
    if activation is None:
        activation = ACT_NONE if Q2 is None else ACT_SILU
    if C is None:
        C = _new((M, N), dtype or X.dtype, X.device, stream)
    elif dtype is not None and dtype != C.dtype:
        raise ValueError("C is not of the given dtype")
    pc, c_type, ldc = _of_shape("C", C, _FLOATS, (M, N), device)
    st = load().sgemm_q4(M, N, K, px, x_type, ldx, pq, ps, pz, p2, ps2, pz2, ldq, lds, group, activation, pc, c_type,
                         ldc, _current_stream(device) if stream is None else _stream(stream))
    if st != SGEMM_OK:
        raise SgemmError(st, "sgemm_q4")
    return C
