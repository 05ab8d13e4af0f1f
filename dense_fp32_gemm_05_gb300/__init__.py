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
    "sgemm_moe", "moe",
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
    lib.sgemm_fp8_plan.argtypes = [i64, i64, i64, i32, ip, ip, ip]
    lib.sgemm_fp8_plan.restype = i32
    lib.sgemm_moe.argtypes = [i64, i64, i64, i64, i64, vp, i32, i64, vp, vp, vp, vp, vp, vp, i64, i64,
                              vp, vp, i64, i64, i32, vp, i64, vp, vp, vp]
    lib.sgemm_moe.restype = i32


def load():
    """Loads the CUDA library (raises if it has not been built)."""
    global _lib
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
            "sgemm_fp8", "sgemm_fp8_plan", "sgemm_moe"]


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


_types = None


def _type_of(dtype):
    """The library's type code of a torch dtype (None: not one of its types)."""
    global _types
    if _types is None:
        import torch
        _types = {torch.float32: TYPE_F32, torch.bfloat16: TYPE_BF16,
                  torch.float8_e4m3fn: TYPE_E4M3, torch.float8_e5m2: TYPE_E5M2}
    return _types.get(dtype)


def _matrix(name, t, types):
    """(address, type, leading dimension) of a 2-D row-major CUDA tensor."""
    code = _type_of(t.dtype)
    if code not in types or not t.is_cuda or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D CUDA tensor of a type the call takes")
    rows, cols = t.shape
    ld, unit = t.stride()
    if cols > 1 and unit != 1:
        raise ValueError(f"{name} must have unit stride along its last dimension")
    return t.data_ptr(), code, (ld if rows > 1 and ld > cols else max(cols, 1))


def _current_stream(device):
    import torch
    return torch.cuda.current_stream(device).cuda_stream


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
    buffers to write into.  Asynchronous on ``stream`` (default: torch's current
    stream on X's device); raises SgemmError on any non-zero status.
    """
    import torch

    px, tx, ldx = _matrix("X", X, (TYPE_F32, TYPE_BF16))
    rows, cols = X.shape
    gr, gc = group
    if Q is None:
        Q = torch.empty((rows, cols), device=X.device, dtype=dtype or torch.float8_e4m3fn)
    elif Q.shape != X.shape or (dtype is not None and dtype != Q.dtype):
        raise ValueError("Q must have X's shape and the given dtype")
    pq, tq, ldq = _matrix("Q", Q, (TYPE_E4M3, TYPE_E5M2))
    row_blocks, col_blocks = (rows + 127) // 128, (cols + 127) // 128
    shape = ((col_blocks, rows) if gr == 1 else
             (row_blocks, cols) if gc == 1 else (row_blocks, col_blocks))
    if S is None:
        S = torch.empty(shape, device=X.device, dtype=torch.float32)
    elif S.shape != shape:
        raise ValueError(f"S must have shape {shape}")
    ps, _, lds = _matrix("S", S, (TYPE_F32,))
    if Q.device != X.device or S.device != X.device:
        raise ValueError("X, Q and S must be on one device")
    st = load().sgemm_fp8_quantize(rows, cols, px, tx, ldx, gr, gc, pq, tq, ldq, ps, lds,
                                   _current_stream(X.device) if stream is None else _stream(stream))
    if st != SGEMM_OK:
        raise SgemmError(st, "sgemm_fp8_quantize")
    return Q, S


def sgemm_fp8(transA, transB, M, N, K, alpha, A, a_type, lda, SA, a_group, ldsa, B, b_type, ldb, SB,
              b_group, ldsb, beta, C, c_type, ldc, stream=None) -> int:
    """C = alpha*op(A)*op(B) + beta*C with quantised A and B; device addresses (int)."""
    return load().sgemm_fp8(_b(transA), _b(transB), M, N, K, alpha, A, a_type, lda, SA, a_group, ldsa,
                            B, b_type, ldb, SB, b_group, ldsb, beta, C, c_type, ldc, _stream(stream))


def sgemm_fp8_plan(M, N, K, num_sms=152):
    """The 8-bit product's tile and cluster size, without a GPU: (status, dict)."""
    outs = [ctypes.c_int(0) for _ in range(3)]
    st = load().sgemm_fp8_plan(M, N, K, num_sms, *[ctypes.byref(o) for o in outs])
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
    Asynchronous on ``stream`` (default: torch's current stream on C's device);
    raises SgemmError on any non-zero status.
    """
    pa, a_type, lda = _matrix("A", A, (TYPE_E4M3, TYPE_E5M2))
    pb, b_type, ldb = _matrix("B", B, (TYPE_E4M3, TYPE_E5M2))
    pc, c_type, ldc = _matrix("C", C, (TYPE_F32, TYPE_BF16))
    psa, _, ldsa = _matrix("SA", SA, (TYPE_F32,))
    psb, _, ldsb = _matrix("SB", SB, (TYPE_F32,))
    ta, tb = transA.upper(), transB.upper()
    M, N = C.shape
    K = A.shape[1] if ta == "N" else A.shape[0]
    kb = (K + 127) // 128
    if A.shape != ((M, K) if ta == "N" else (K, M)) or B.shape != ((K, N) if tb == "N" else (N, K)):
        raise ValueError("the shapes of A, B and C do not fit together")

    def blocks(t):
        return ((t.shape[0] + 127) // 128, (t.shape[1] + 127) // 128)

    if SA.shape != ((kb, M) if a_group == 1 else blocks(A)) or \
            SB.shape != ((kb, N) if b_group == 1 else blocks(B)):
        raise ValueError("the scales' shapes do not fit the operands and their groups")
    device = C.device
    if not (A.device == B.device == SA.device == SB.device == device):
        raise ValueError("the operands must be on one device")
    st = load().sgemm_fp8(ta.encode(), tb.encode(), M, N, K, alpha, pa, a_type, lda, psa, a_group, ldsa,
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


def _experts(name, t, E, rows, cols):
    """(address, row stride, matrix stride) of E matrices of E4M3 codes."""
    if _type_of(t.dtype) != TYPE_E4M3 or not t.is_cuda or t.shape != (E, rows, cols) or t.stride(2) != 1:
        raise ValueError(f"{name} must be an {E} x {rows} x {cols} CUDA tensor of float8_e4m3fn codes "
                         "with unit stride along its last dimension")
    stride, ld, _ = t.stride()
    return t.data_ptr(), ld, stride


def _packed(name, t, shape, dtype):
    if t.shape != shape or t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor of shape {shape}")
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
    weights take buffers to write into.  Asynchronous on ``stream`` (default:
    torch's current stream on x's device); raises SgemmError on any non-zero
    status.
    """
    import torch

    px, x_type, ldx = _matrix("x", x, (TYPE_F32, TYPE_BF16))
    T, D = x.shape
    E, F = gate.shape[:2]
    device = x.device
    pg, ld_in, stride_in = _experts("gate", gate, E, F, D)
    pu, ld_up, stride_up = _experts("up", up, E, F, D)
    pd, ld_down, stride_down = _experts("down", down, E, D, F)
    if (ld_up, stride_up) != (ld_in, stride_in):
        raise ValueError("gate and up must have the same strides")
    fb, db = (F + 127) // 128, (D + 127) // 128
    f32 = torch.float32
    if router is None and logits is None:
        raise ValueError("give router or logits")
    pr = _packed("router", router, (E, D), f32) if router is not None else None
    if logits is None:
        logits = torch.empty((T, E), device=device, dtype=f32)
    if y is None:
        y = torch.empty((T, D), device=device, dtype=x.dtype)
    elif y.shape != x.shape or y.dtype != x.dtype:
        raise ValueError("y must have x's shape and dtype")
    if indices is None:
        indices = torch.empty((T, topk), device=device, dtype=torch.int32)
    if weights is None:
        weights = torch.empty((T, topk), device=device, dtype=f32)
    py, _, ldy = _matrix("y", y, (TYPE_F32, TYPE_BF16))
    for t in (router, logits, gate, s_gate, up, s_up, down, s_down, y, indices, weights):
        if t is not None and t.device != device:
            raise ValueError("the operands must be on one device")
    st = load().sgemm_moe(
        T, D, F, E, topk, px, x_type, ldx, pr, _packed("logits", logits, (T, E), f32), pg,
        _packed("s_gate", s_gate, (E, fb, db), f32), pu, _packed("s_up", s_up, (E, fb, db), f32), ld_in,
        stride_in, pd, _packed("s_down", s_down, (E, db, fb), f32), ld_down, stride_down,
        int(renormalize), py, ldy, _packed("indices", indices, (T, topk), torch.int32),
        _packed("weights", weights, (T, topk), f32),
        _current_stream(device) if stream is None else _stream(stream))
    if st != SGEMM_OK:
        raise SgemmError(st, "sgemm_moe")
    return y, logits, indices, weights
