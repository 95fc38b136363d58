"""Python binding of libgemm_nt: Out = A @ B.T, fp16 inputs, fp32 accumulate/output.

The functions named like the C ABI (include/gemm_nt.h) take raw device
pointers and sizes and only marshal arguments; ``gemm_nt`` and
``gemm_nt_batched`` do the same for torch CUDA tensors (pointers, strides and
the current stream).  Every step of the product runs in the library's CUDA
kernels.  There is no fallback: if libgemm_nt.so has not been built, or a call
fails, an exception is raised.
"""
import ctypes
import enum
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libgemm_nt.so")


class Status(enum.IntEnum):
    OK = 0
    INVALID_VALUE = 1
    MISALIGNED = 2          # reserved: never returned
    OVERLAP = 3
    LAUNCH = 4
    DEVICE_TIMEOUT = 5
    UNSUPPORTED_DEVICE = 6
    NOT_SUPPORTED = 7
    SCRATCH_TOO_SMALL = 8


class DType(enum.IntEnum):
    F16 = 0
    BF16 = 1
    F32 = 2
    E4M3 = 3  # 8-bit floats (A and B only)
    E5M2 = 4
    E2M3 = 5  # 6- and 4-bit floats, packed along K, little-endian bits (A and B only)
    E3M2 = 6
    E2M1 = 7


class Major(enum.IntEnum):
    K = 0   # operand (rows, K) stored row-major
    MN = 1  # operand stored as its transpose, (K, rows) row-major


class Path(enum.IntEnum):
    AUTO = 0
    TC05 = 1
    SKINNY = 2
    MMASYNC = 3
    TC05_PAIR = 4
    TC05_M64 = 5   # 64-row tiles, plain M = 64 MMA
    TC05_WS = 6    # 32- or 64-row tiles, weight-stationary MMA


class GemmError(RuntimeError):
    def __init__(self, status):
        self.status = Status(status)
        super().__init__("libgemm_nt: %s (%s)" % (error_string(status), self.status.name))


class Scale128(ctypes.Structure):
    """gemm_scale128_t: fp32 scales of one operand, one for each 128 elements of
    K of every row (rows = 1) or of every 128 rows (rows = 128)."""
    _fields_ = [("data", ctypes.c_void_p), ("rows", ctypes.c_int32), ("row_stride", ctypes.c_int64),
                ("kb_stride", ctypes.c_int64), ("batch_stride", ctypes.c_int64)]


# name -> (restype, argtypes); mirrors include/gemm_nt.h
_i64, _vp, _u64 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_uint64
_sp = ctypes.POINTER(Scale128)
_SIGNATURES = {
    "gemm_nt_f16_f32": (ctypes.c_int, [_vp, _vp, _vp] + [_i64] * 6 + [_vp]),
    "gemm_nt_f16_f32_batched": (ctypes.c_int, [_vp, _vp, _vp] + [_i64] * 10 + [_vp]),
    "gemm_nt_f16_f32_batched_path": (ctypes.c_int, [_vp, _vp, _vp] + [_i64] * 10 + [ctypes.c_int, _vp]),
    "gemm_nt_f16_f32_from_host": (ctypes.c_int, [_vp] * 6 + [_i64] * 4 + [_vp]),
    "gemm_nt_f16_f32_batched_no_alloc": (ctypes.c_int, [_vp, _vp, _vp] + [_i64] * 10 + [_vp]),
    "gemm_nt_batched_ex": (ctypes.c_int, [_vp, _vp, _vp, ctypes.c_int, ctypes.c_int] + [_i64] * 10
                           + [ctypes.c_int, _vp]),
    "gemm_nt_batched_major": (ctypes.c_int, [_vp, ctypes.c_int, _vp, ctypes.c_int, _vp, ctypes.c_int, ctypes.c_int]
                              + [_i64] * 10 + [ctypes.c_int, _vp]),
    "gemm_nt_mx": (ctypes.c_int, [_vp] * 5 + [ctypes.c_int, ctypes.c_int] + [_i64] * 10 + [ctypes.c_int, _vp]),
    "gemm_nt_mx_scale_bytes": (_i64, [_i64, _i64]),
    "gemm_nt_mx_pack_scales": (ctypes.c_int, [_vp, _i64, _i64, _vp, _i64, _i64, _i64, _vp]),
    "gemm_nt_block128": (ctypes.c_int, [_vp, _sp, _vp, _sp, _vp, ctypes.c_int, ctypes.c_int] + [_i64] * 10
                         + [ctypes.c_int, _vp]),
    "gemm_nt_block128_quantize": (ctypes.c_int, [_vp, ctypes.c_int, _i64, _i64, _i64, _vp, _i64, _sp, _vp, _i64, _sp,
                                                 ctypes.c_int, _vp]),
    "gemm_nt_moe": (ctypes.c_int, [_vp, _i64, _vp, _i64, _vp, _i64, _i64, _sp, _vp, _i64, _i64, _sp, _vp, _i64,
                                   ctypes.c_int, ctypes.c_int] + [_i64] * 5 + [ctypes.c_int, _vp, _i64, _vp]),
    "gemm_nt_moe_workspace_bytes": (_i64, [_i64, _i64, _i64]),
    "gemm_nt_select_path": (ctypes.c_int, [_vp, _vp, _vp] + [_i64] * 10),
    "gemm_nt_check": (ctypes.c_int, [_vp]),
    "gemm_nt_error_string": (ctypes.c_char_p, [ctypes.c_int]),
    "gemm_nt_probe_m16n8k16": (ctypes.c_int, [_vp] * 6),
    "gemm_nt_debug_set_wait_limit": (None, [_u64]),
    "gemm_nt_debug_set_fault": (None, [ctypes.c_int]),
}

_lib = None


def load(path=LIB_PATH):
    """Load libgemm_nt.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise RuntimeError(
                "libgemm_nt.so is not built (%s); run `python -m dense_fp16_tensor_gemm_gb300._build`"
                % path)
        lib = ctypes.CDLL(path)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def _check(status):
    if status != 0:
        raise GemmError(status)


def error_string(status):
    return load().gemm_nt_error_string(int(status)).decode()


# ---------------------------------------------------------------- C-ABI mirror
def gemm_nt_f16_f32(A, B, Out, M, N, K, lda, ldb, ldo, stream=0):
    _check(load().gemm_nt_f16_f32(A, B, Out, M, N, K, lda, ldb, ldo, stream))


def gemm_nt_f16_f32_batched(A, B, Out, M, N, K, lda, ldb, ldo, strideA, strideB, strideO, batch,
                            stream=0):
    _check(load().gemm_nt_f16_f32_batched(A, B, Out, M, N, K, lda, ldb, ldo, strideA, strideB,
                                          strideO, batch, stream))


def gemm_nt_f16_f32_batched_path(A, B, Out, M, N, K, lda, ldb, ldo, strideA, strideB, strideO,
                                 batch, path, stream=0):
    _check(load().gemm_nt_f16_f32_batched_path(A, B, Out, M, N, K, lda, ldb, ldo, strideA, strideB,
                                               strideO, batch, int(path), stream))


def gemm_nt_batched_ex(A, B, Out, ab_type, out_type, M, N, K, lda, ldb, ldo, strideA, strideB, strideO,
                       batch, path=0, stream=0):
    _check(load().gemm_nt_batched_ex(A, B, Out, int(ab_type), int(out_type), M, N, K, lda, ldb, ldo,
                                     strideA, strideB, strideO, batch, int(path), stream))


def gemm_nt_batched_major(A, a_major, B, b_major, Out, ab_type, out_type, M, N, K, lda, ldb, ldo, strideA,
                          strideB, strideO, batch, path=0, stream=0):
    _check(load().gemm_nt_batched_major(A, int(a_major), B, int(b_major), Out, int(ab_type), int(out_type), M, N,
                                        K, lda, ldb, ldo, strideA, strideB, strideO, batch, int(path), stream))


def gemm_nt_mx(A, SA, B, SB, Out, ab_type, out_type, M, N, K, lda, ldb, ldo, strideA, strideB, strideO, batch,
               path=0, stream=0):
    """Block-scaled 8-bit product; SA / SB in the packed atom layout (see
    include/gemm_nt.h)."""
    _check(load().gemm_nt_mx(A, SA, B, SB, Out, int(ab_type), int(out_type), M, N, K, lda, ldb, ldo, strideA,
                             strideB, strideO, batch, int(path), stream))


def gemm_nt_mx_scale_bytes(rows, K):
    return int(load().gemm_nt_mx_scale_bytes(rows, K))


def gemm_nt_mx_pack_scales(plain, ld, stride, packed, rows, K, batch=1, stream=0):
    _check(load().gemm_nt_mx_pack_scales(plain, ld, stride, packed, rows, K, batch, stream))


def gemm_nt_block128(A, SA, B, SB, Out, ab_type, out_type, M, N, K, lda, ldb, ldo, strideA, strideB, strideO, batch,
                     path=0, stream=0):
    """8-bit product with an fp32 scale per 128 elements of K; SA / SB are
    Scale128 (or None when K is 0)."""
    _check(load().gemm_nt_block128(A, SA, B, SB, Out, int(ab_type), int(out_type), M, N, K, lda, ldb, ldo, strideA,
                                   strideB, strideO, batch, int(path), stream))


def gemm_nt_block128_quantize(X, x_type, rows, cols, ldx, Q, ldq, SQ, QT, ldqt, ST, q_type, stream=0):
    _check(load().gemm_nt_block128_quantize(X, int(x_type), rows, cols, ldx, Q, ldq, SQ, QT, ldqt, ST, int(q_type),
                                            stream))


def gemm_nt_moe(X, ldx, logits, ldl, W13, ldw13, strideW13, S13, W2, ldw2, strideW2, S2, Out, ldo, x_type, w_type,
                tokens, experts, topk, hidden, inner, renormalize, workspace, workspace_bytes, stream=0):
    _check(load().gemm_nt_moe(X, ldx, logits, ldl, W13, ldw13, strideW13, S13, W2, ldw2, strideW2, S2, Out, ldo,
                              int(x_type), int(w_type), tokens, experts, topk, hidden, inner, int(renormalize),
                              workspace, workspace_bytes, stream))


def gemm_nt_moe_workspace_bytes(tokens, topk, inner):
    return int(load().gemm_nt_moe_workspace_bytes(tokens, topk, inner))


def gemm_nt_f16_f32_batched_no_alloc(A, B, Out, M, N, K, lda, ldb, ldo, strideA, strideB, strideO,
                                     batch, stream=0):
    """The batched product without any device allocation (fixed scratch array
    inside the library; see include/gemm_nt.h)."""
    _check(load().gemm_nt_f16_f32_batched_no_alloc(A, B, Out, M, N, K, lda, ldb, ldo, strideA, strideB,
                                                   strideO, batch, stream))


def gemm_nt_f16_f32_from_host(A_host, B_host, Out_host, dA, dB, dOut, M, N, K, batch, stream=0):
    _check(load().gemm_nt_f16_f32_from_host(A_host, B_host, Out_host, dA, dB, dOut, M, N, K, batch,
                                            stream))


def gemm_nt_select_path(A, B, Out, M, N, K, lda, ldb, ldo, strideA=0, strideB=0, strideO=0, batch=1):
    return Path(load().gemm_nt_select_path(A, B, Out, M, N, K, lda, ldb, ldo, strideA, strideB,
                                           strideO, batch))


def gemm_nt_check(stream=0):
    _check(load().gemm_nt_check(stream))


def gemm_nt_probe_m16n8k16(A, B, ar, br, dr, stream=0):
    _check(load().gemm_nt_probe_m16n8k16(A, B, ar, br, dr, stream))


def gemm_nt_debug_set_wait_limit(cycles):
    load().gemm_nt_debug_set_wait_limit(int(cycles))


def gemm_nt_debug_set_fault(fault):
    load().gemm_nt_debug_set_fault(int(fault))


# ---------------------------------------------------------------- torch tensors
def _stream_handle(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _matrix_ld(t, name):
    if t.stride(-1) != 1:
        raise ValueError("%s must have unit stride along its last dimension" % name)
    return t.stride(-2) if t.shape[-2] > 1 else max(t.shape[-1], 1)


def _dtypes(A, B, out, out_dtype):
    import torch
    codes = {torch.float16: DType.F16, torch.bfloat16: DType.BF16, torch.float32: DType.F32,
             torch.float8_e4m3fn: DType.E4M3, torch.float8_e5m2: DType.E5M2}
    if A.dtype != B.dtype or A.dtype not in (torch.float16, torch.bfloat16, torch.float8_e4m3fn,
                                             torch.float8_e5m2):
        raise TypeError("A and B must have the same type: float16, bfloat16, float8_e4m3fn or float8_e5m2")
    dt = out.dtype if out is not None else (out_dtype or torch.float32)
    if dt not in (torch.float32, torch.float16, torch.bfloat16):
        raise TypeError("out must be float32, float16 or bfloat16")
    return codes[A.dtype], codes[dt], dt


def gemm_nt(A, B, out=None, path=Path.AUTO, stream=None, out_dtype=None):
    """Out = A @ B.T for torch CUDA tensors A (M,K), B (N,K), both fp16 or both
    bf16, accumulated in fp32.

    Row strides may exceed the row length; the last dimension must be
    contiguous.  ``out`` (M,N) is allocated if not given, as ``out_dtype``
    (default float32; float16 or bfloat16 round to nearest even).  Runs on
    ``stream`` (default: torch's current stream) as under ``torch.cuda.stream``,
    allocations included.
    """
    side = _elsewhere(stream)
    if side is not None:
        return _run_on(side, gemm_nt, A, B, out, path, None, out_dtype, given=out)
    import torch
    if A.dim() != 2 or B.dim() != 2 or A.shape[1] != B.shape[1]:
        raise ValueError("shapes: A (M,K), B (N,K)")
    ab, ot, dt = _dtypes(A, B, out, out_dtype)
    M, K = A.shape
    N = B.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=dt, device=A.device)
    if tuple(out.shape) != (M, N):
        raise ValueError("out must have shape (M,N)")
    gemm_nt_batched_ex(A.data_ptr(), B.data_ptr(), out.data_ptr(), ab, ot, M, N, K,
                       _matrix_ld(A, "A"), _matrix_ld(B, "B"), _matrix_ld(out, "out"),
                       0, 0, 0, 1, path, _stream_handle(stream))
    return out


def pack_mx_scales(S, K, stream=None):
    """Plain block scales -> the packed atom layout, on the device: S a uint8
    CUDA tensor (rows, ceil(K/32)) or (batch, rows, ceil(K/32)) of E8M0
    bytes, last dimension contiguous.  Returns a new uint8 tensor."""
    side = _elsewhere(stream)
    if side is not None:
        return _run_on(side, pack_mx_scales, S, K)
    import torch
    if S.dtype != torch.uint8 or S.dim() not in (2, 3) or S.stride(-1) != 1:
        raise ValueError("S: uint8 (rows, ceil(K/32)) or (batch, rows, ceil(K/32)), last dimension contiguous")
    S3 = S if S.dim() == 3 else S[None]
    batch, rows, kb = S3.shape
    if kb != (K + 31) // 32:
        raise ValueError("S has %d scale columns, K=%d needs %d" % (kb, K, (K + 31) // 32))
    packed = torch.empty(batch * gemm_nt_mx_scale_bytes(rows, K), dtype=torch.uint8, device=S.device)
    gemm_nt_mx_pack_scales(S3.data_ptr(), S3.stride(1), S3.stride(0), packed.data_ptr(), rows, K, batch,
                           _stream_handle(stream))
    return packed


def gemm_nt_mx_tensors(A, SA, B, SB, out=None, path=Path.AUTO, stream=None, out_dtype=None):
    """Block-scaled Out = (A * sa) @ (B * sb).T for torch CUDA tensors: A (M,K)
    and B (N,K) both float8_e4m3fn or both float8_e5m2; SA (M, ceil(K/32))
    and SB (N, ceil(K/32)) uint8 E8M0 scales (2^(e-127)), one per 32
    consecutive K elements of a row, in the plain layout (packed here).
    ``out``/``out_dtype`` as in :func:`gemm_nt`."""
    side = _elsewhere(stream)
    if side is not None:
        return _run_on(side, gemm_nt_mx_tensors, A, SA, B, SB, out, path, None, out_dtype, given=out)
    import torch
    if A.dim() != 2 or B.dim() != 2 or A.shape[1] != B.shape[1]:
        raise ValueError("shapes: A (M,K), B (N,K)")
    ab, ot, dt = _dtypes(A, B, out, out_dtype)
    if ab not in (DType.E4M3, DType.E5M2):
        raise TypeError("block-scaled inputs are float8_e4m3fn or float8_e5m2")
    M, K = A.shape
    N = B.shape[0]
    pa, pb = pack_mx_scales(SA, K, stream), pack_mx_scales(SB, K, stream)
    if out is None:
        out = torch.empty((M, N), dtype=dt, device=A.device)
    if tuple(out.shape) != (M, N):
        raise ValueError("out must have shape (M,N)")
    gemm_nt_mx(A.data_ptr(), pa.data_ptr(), B.data_ptr(), pb.data_ptr(), out.data_ptr(), ab, ot, M, N, K,
               _matrix_ld(A, "A"), _matrix_ld(B, "B"), _matrix_ld(out, "out"), 0, 0, 0, 1, path,
               _stream_handle(stream))
    return out


PACKED_BITS = {DType.E2M3: 6, DType.E3M2: 6, DType.E2M1: 4}


def gemm_nt_packed(A, B, K, ab_dtype, SA=None, SB=None, out=None, path=Path.AUTO, stream=None, out_dtype=None):
    """Out = A @ B.T for 6- or 4-bit float inputs stored packed: A (M, K*w/8)
    and B (N, K*w/8) uint8 CUDA tensors (w = 6 for E2M3 / E3M2, 4 for E2M1),
    element k of a row at bits [w*k, w*k+w) of the row, little-endian.  K is a
    multiple of 128, rows start on 32-byte boundaries.  With SA (M, K/32) and
    SB (N, K/32) uint8 E8M0 scales (plain layout) the product is block-scaled
    as in :func:`gemm_nt_mx_tensors`.  ``out``/``out_dtype`` as in :func:`gemm_nt`."""
    side = _elsewhere(stream)
    if side is not None:
        return _run_on(side, gemm_nt_packed, A, B, K, ab_dtype, SA, SB, out, path, None, out_dtype, given=out)
    import torch
    ab = DType(ab_dtype)
    if ab not in PACKED_BITS:
        raise TypeError("ab_dtype must be E2M3, E3M2 or E2M1")
    bits = PACKED_BITS[ab]
    if A.dim() != 2 or B.dim() != 2 or A.dtype != torch.uint8 or B.dtype != torch.uint8:
        raise TypeError("A and B are 2-D uint8 tensors of packed elements")
    if K * bits % 8 or A.shape[1] != K * bits // 8 or B.shape[1] != K * bits // 8:
        raise ValueError("A and B must hold K packed elements per row")
    if (SA is None) != (SB is None):
        raise ValueError("give both SA and SB, or neither")
    dt = out.dtype if out is not None else (out_dtype or torch.float32)
    ocodes = {torch.float32: DType.F32, torch.float16: DType.F16, torch.bfloat16: DType.BF16}
    if dt not in ocodes:
        raise TypeError("out must be float32, float16 or bfloat16")
    M, N = A.shape[0], B.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=dt, device=A.device)
    if tuple(out.shape) != (M, N):
        raise ValueError("out must have shape (M,N)")
    # pitches in elements: the byte pitch of a row times 8 / w
    pa_bytes, pb_bytes = _matrix_ld(A, "A"), _matrix_ld(B, "B")
    if pa_bytes * 8 % bits or pb_bytes * 8 % bits:
        raise ValueError("row pitches must hold whole packing groups")
    lda, ldb = pa_bytes * 8 // bits, pb_bytes * 8 // bits
    if SA is None:
        gemm_nt_batched_ex(A.data_ptr(), B.data_ptr(), out.data_ptr(), ab, ocodes[dt], M, N, K, lda, ldb,
                           _matrix_ld(out, "out"), 0, 0, 0, 1, path, _stream_handle(stream))
    else:
        pa, pb = pack_mx_scales(SA, K, stream), pack_mx_scales(SB, K, stream)
        gemm_nt_mx(A.data_ptr(), pa.data_ptr(), B.data_ptr(), pb.data_ptr(), out.data_ptr(), ab, ocodes[dt], M, N,
                   K, lda, ldb, _matrix_ld(out, "out"), 0, 0, 0, 1, path, _stream_handle(stream))
    return out


def gemm_nt_batched(A, B, out=None, path=Path.AUTO, stream=None, out_dtype=None):
    """Out[b] = A[b] @ B[b].T for torch CUDA tensors A (batch,M,K), B (batch,N,K),
    both fp16 or both bf16 (a batch stride of 0, e.g. from ``expand``, shares
    the operand); ``out``/``out_dtype`` as in :func:`gemm_nt`."""
    side = _elsewhere(stream)
    if side is not None:
        return _run_on(side, gemm_nt_batched, A, B, out, path, None, out_dtype, given=out)
    import torch
    if A.dim() != 3 or B.dim() != 3 or A.shape[0] != B.shape[0] or A.shape[2] != B.shape[2]:
        raise ValueError("shapes: A (batch,M,K), B (batch,N,K)")
    ab, ot, dt = _dtypes(A, B, out, out_dtype)
    batch, M, K = A.shape
    N = B.shape[1]
    if out is None:
        out = torch.empty((batch, M, N), dtype=dt, device=A.device)
    if tuple(out.shape) != (batch, M, N):
        raise ValueError("out must have shape (batch,M,N)")
    gemm_nt_batched_ex(A.data_ptr(), B.data_ptr(), out.data_ptr(), ab, ot, M, N, K,
                       _matrix_ld(A, "A"), _matrix_ld(B, "B"), _matrix_ld(out, "out"),
                       A.stride(0), B.stride(0), out.stride(0), batch, path, _stream_handle(stream))
    return out


# ---------------------------------------------------------------- one scale per block of 128
# These calls serve single tokens, where the host's time per call counts: types
# are looked up once, the stream handle is read without building a Stream object,
# and an output is one allocation.  With `stream` they run as under
# torch.cuda.stream(stream), allocations included.
_torch = None
_CODES = {}     # torch dtype -> gemm_dtype_t value
_IN_F8 = _OUT = _X16 = ()


def _init_torch():
    global _torch, _IN_F8, _OUT, _X16
    import torch
    _CODES.update({torch.float16: 0, torch.bfloat16: 1, torch.float32: 2, torch.float8_e4m3fn: 3,
                   torch.float8_e5m2: 4})
    _IN_F8 = (torch.float8_e4m3fn, torch.float8_e5m2)
    _OUT = (torch.float32, torch.float16, torch.bfloat16)
    _X16 = (torch.float16, torch.bfloat16)
    _torch = torch
    return torch


def _one_of(dtype, allowed, what):
    if dtype not in allowed:
        raise TypeError("%s must be one of %s" % (what, ", ".join(str(a).replace("torch.", "") for a in allowed)))
    return _CODES[dtype]


def _same_device(first, *others):
    """The index of the CUDA device that all of a call's tensors (None: not given) lie on,
    torch's current one: the library reads their addresses there.  (Indexes, and torch's
    own current index: device objects and torch.cuda.current_device() took 4 us a call.)"""
    index = first.get_device()
    if index < 0:
        raise ValueError("tensors must be on a CUDA device, not %s" % first.device)
    for t in others:
        if t is not None and t.get_device() != index:
            raise ValueError("tensors on %s and %s in one call" % (first.device, t.device))
    if index != _torch._C._cuda_getDevice():
        raise ValueError("tensors on %s, which is not the current device" % first.device)
    return index


def _stream_of(index):
    """The handle of torch's current stream on the device of that index."""
    return _torch._C._cuda_getCurrentRawStream(index)


def _elsewhere(stream):
    """`stream` as a torch stream if it is another than torch's current one, else None."""
    if stream is None:
        return None
    cuda, handle = (_torch or _init_torch()).cuda, _stream_handle(stream)
    if handle == cuda.current_stream().cuda_stream:
        return None
    if isinstance(stream, cuda.Stream):
        return stream
    return cuda.ExternalStream(handle) if handle else cuda.default_stream()


def _record(result, stream, given):
    """Keeps the tensors of a call's result, but for the caller's own `given`, from
    being handed out again before what `stream` holds when they are freed is done."""
    if isinstance(result, tuple):
        for r in result:
            _record(r, stream, given)
    elif result is not given:
        result.record_stream(stream)


def _run_on(side, call, *args, given=None):
    """call(*args) with `side` as torch's current stream, so that its temporaries and
    results come from side's memory: a block of the caller's current stream may still
    be in use by work queued there, which side does not wait for.  The results are
    recorded for the caller's stream, which will read them."""
    caller = _torch.cuda.current_stream()
    with _torch.cuda.stream(side):
        result = call(*args)
    _record(result, caller, given)
    return result


def _pitch(shape, strides, name):
    """As _matrix_ld, from a tensor's shape and strides."""
    if strides[-1] != 1:
        raise ValueError("%s must have unit stride along its last dimension" % name)
    return strides[-2] if shape[-2] > 1 else max(shape[-1], 1)


def _scale128(S, rows, K, name):
    """A scale tensor (rows or ceil(rows/128), ceil(K/128)), optionally with a
    leading batch dimension, as the C struct."""
    if S.dtype != _torch.float32:
        raise TypeError("%s must be float32" % name)
    shape, strides = S.shape, S.stride()
    n, kb = shape[-2], (K + 127) // 128
    if len(shape) not in (2, 3) or shape[-1] != kb or n not in (rows, (rows + 127) // 128):
        raise ValueError("%s: (%d or %d, %d) scales for %d rows and K = %d"
                         % (name, rows, (rows + 127) // 128, kb, rows, K))
    return Scale128(S.data_ptr(), 1 if n == rows else 128, strides[-2], strides[-1],
                    strides[0] if len(shape) == 3 and shape[0] > 1 else 0)


def gemm_nt_block128_tensors(A, SA, B, SB, out=None, path=Path.AUTO, stream=None, out_dtype=None):
    """Out[i,j] = sum_c SA[i,c] SB[j,c] sum_{k in block c} A[i,k] B[j,k] for torch
    CUDA tensors, c the blocks of 128 of K: A (M,K) and B (N,K) both
    float8_e4m3fn or both float8_e5m2; SA and SB float32, one scale a row (M or
    N, ceil(K/128)) or one for 128 rows (ceil(M/128) or ceil(N/128),
    ceil(K/128)), any strides.  With a leading batch dimension on all four
    (stride 0 shares an operand), a batch of products.  ``out``/``out_dtype`` as
    in :func:`gemm_nt`, float32 by default.
    """
    side = _elsewhere(stream)
    if side is not None:
        return _run_on(side, gemm_nt_block128_tensors, A, SA, B, SB, out, path, None, out_dtype, given=out)
    torch = _torch or _init_torch()
    ash, bsh = A.shape, B.shape
    dims = len(ash)
    batched = dims == 3
    if not (batched or dims == 2) or len(bsh) != dims or ash[-1] != bsh[-1] or SA.dim() != dims \
            or SB.dim() != dims or batched and not ash[0] == bsh[0] == SA.shape[0] == SB.shape[0]:
        raise ValueError("shapes: A (M,K), B (N,K) and their scales, or the same with a leading batch dimension")
    if A.dtype != B.dtype:
        raise TypeError("A and B must have the same type")
    ab = _one_of(A.dtype, _IN_F8, "A and B")
    dt = out.dtype if out is not None else (out_dtype or torch.float32)
    ot = _one_of(dt, _OUT, "out")
    M, K = ash[-2:]
    N = bsh[-2]
    shape = (ash[0], M, N) if batched else (M, N)
    sa, sb = _scale128(SA, M, K, "SA"), _scale128(SB, N, K, "SB")
    index = _same_device(A, SA, B, SB, out)
    if out is None:
        out = torch.empty(shape, dtype=dt, device=A.device)
    elif tuple(out.shape) != shape:
        raise ValueError("out must have shape (M,N), with A's batch dimension")
    ast, bst, ost = A.stride(), B.stride(), out.stride()
    gemm_nt_block128(A.data_ptr(), sa, B.data_ptr(), sb, out.data_ptr(), ab, ot, M, N, K,
                     _pitch(ash, ast, "A"), _pitch(bsh, bst, "B"), _pitch(shape, ost, "out"),
                     ast[0] if batched else 0, bst[0] if batched else 0, ost[0] if batched else 0,
                     ash[0] if batched else 1, path, _stream_of(index))
    return out


def _quantized(rows, cols, q_dtype, block_rows, device):
    """Empty codes and scales for a (rows, cols) matrix, the codes' pitch, and
    the scales as the C struct.  Rows of codes, and columns of single rows'
    scales, start on 16-byte boundaries, as the products read them fastest."""
    pitch, kb = (cols + 15) // 16 * 16, (cols + 127) // 128
    q = _torch.empty_strided((rows, cols), (pitch, 1), dtype=q_dtype, device=device)
    if block_rows == 1:
        n, strides = rows, (1, (rows + 3) // 4 * 4)
    else:
        n, strides = (rows + 127) // 128, (kb, 1)
    s = _torch.empty_strided((n, kb), strides, dtype=_torch.float32, device=device)
    return q, s, pitch, Scale128(s.data_ptr(), block_rows, strides[0], strides[1], 0)


def quantize_block128(X, q_dtype=None, block_rows=1, transposed=False, stream=None):
    """8-bit codes and fp32 scales of X (rows, cols; float32, float16 or
    bfloat16), one scale for each 1 x 128 (``block_rows`` 1) or 128 x 128 (128)
    block: a = max(max |x|, 2^-100), scale = a * (1/F), code = x * (F * (1/a))
    rounded to ``q_dtype`` (float8_e4m3fn by default, or float8_e5m2), F its
    largest value.

    Returns ``(Q, S)``, or with ``transposed`` ``(Q, S, QT, ST)`` from one read
    of X: QT (cols, rows) is X transposed, quantised in blocks of its own rows.
    Rows of the codes start on 16-byte boundaries; scales of single rows are
    stored with the rows adjacent.
    """
    side = _elsewhere(stream)
    if side is not None:
        return _run_on(side, quantize_block128, X, q_dtype, block_rows, transposed)
    q, s, _, qt, st, _ = _quantize(X, q_dtype, block_rows, transposed)
    return (q, s, qt, st) if transposed else (q, s)


def _quantize(X, q_dtype, block_rows, transposed, beside=()):
    """The work of quantize_block128: Q, S and S as the C struct, and the same
    of X transposed.  `beside`: what the caller's next calls read on X's device."""
    torch = _torch or _init_torch()
    shape = X.shape
    if len(shape) != 2:
        raise ValueError("X must be a matrix")
    if block_rows not in (1, 128):
        raise ValueError("block_rows must be 1 or 128")
    q_dtype = q_dtype or torch.float8_e4m3fn
    code = _one_of(q_dtype, _IN_F8, "q_dtype")
    xt = _one_of(X.dtype, _OUT, "X")
    ldx = _pitch(shape, X.stride(), "X")
    rows, cols = shape
    index, device = _same_device(X, *beside), X.device
    q, s, ldq, sq = _quantized(rows, cols, q_dtype, block_rows, device)
    qt, st, ldqt, sqt = _quantized(cols, rows, q_dtype, block_rows, device) if transposed else (None, None, 0, None)
    gemm_nt_block128_quantize(X.data_ptr(), xt, rows, cols, ldx, q.data_ptr(), ldq, sq, qt.data_ptr() if transposed else 0,
                              ldqt, sqt, code, _stream_of(index))
    return q, s, sq, qt, st, sqt


def _product(A, SA, B, SB, dtype):
    """A @ B.T of two matrices of codes whose scales are C structs."""
    (M, K), (N, _) = A.shape, B.shape
    out = _torch.empty((M, N), dtype=dtype, device=A.device)
    gemm_nt_block128(A.data_ptr(), SA, B.data_ptr(), SB, out.data_ptr(), _CODES[A.dtype], _CODES[dtype], M, N, K,
                     _pitch((M, K), A.stride(), "A"), _pitch((N, K), B.stride(), "B"), max(N, 1), 0, 0, 0, 1, 0,
                     _stream_of(A.get_device()))
    return out


def _weight(W, SW, width, name):
    """Checks a matrix of codes against the columns it multiplies; its scales as
    the C struct."""
    _torch or _init_torch()
    if W.dim() != 2 or SW.dim() != 2 or W.shape[1] != width:
        raise ValueError("%s must be a matrix with %d columns, with its scales" % (name, width))
    return _scale128(SW, W.shape[0], width, "S" + name)


def linear_block128(X, W, SW, stream=None):
    """Y = X @ W.T in 8 bits: X (tokens, in) float16 or bfloat16 is quantised by
    rows; W (out, in) float8_e4m3fn with scales SW (ceil(out/128), ceil(in/128)),
    as ``quantize_block128(weight, block_rows=128)`` leaves it.  Returns Y in X's
    type and what :func:`linear_block128_backward` needs (X transposed, in 8
    bits)."""
    side = _elsewhere(stream)
    if side is not None:
        return _run_on(side, linear_block128, X, W, SW)
    if X.dim() != 2:
        raise ValueError("X must be a matrix")
    sw = _weight(W, SW, X.shape[1], "W")
    q, s, sq, qt, st, _ = _quantize(X, W.dtype, 1, True, (W, SW))  # s, which sq points into, stays until the product is launched
    return _product(q, sq, W, sw, X.dtype), (qt, st)


def linear_block128_backward(dY, saved, WT, SWT, stream=None):
    """Gradients of :func:`linear_block128`: dX = dY @ W in dY's type and dW =
    dY.T @ X in float32, both products in 8 bits.  WT (in, out) and SWT are W's
    codes and scales transposed (the ``transposed`` half of
    ``quantize_block128(weight, block_rows=128, transposed=True)``)."""
    side = _elsewhere(stream)
    if side is not None:
        _record(tuple(saved), side, None)
        return _run_on(side, linear_block128_backward, dY, saved, WT, SWT)
    if dY.dim() != 2:
        raise ValueError("dY must be a matrix")
    qt_x, st_x = saved
    tokens, width = dY.shape
    sw, sx = _weight(WT, SWT, width, "WT"), _weight(qt_x, st_x, tokens, "XT")
    if qt_x.dtype != WT.dtype:
        raise TypeError("the weights' and the saved codes' types differ")
    q, s, sq, qt, st, sqt = _quantize(dY, WT.dtype, 1, True, (WT, SWT, qt_x, st_x))
    return _product(q, sq, WT, sw, dY.dtype), _product(qt, sqt, qt_x, sx, _torch.float32)


_MOE_SHAPES = ("shapes: X (tokens, hidden), logits (tokens, experts), W13 (experts, 2*inner, hidden), "
               "W2 (experts, hidden, inner)")


def moe_few_tokens(X, logits, W13, W2, topk, S13=None, S2=None, renormalize=True, out=None, workspace=None,
                   stream=None):
    """A mixture-of-experts layer for up to 128 tokens (see gemm_nt_moe in
    include/gemm_nt.h): X (tokens, hidden) float16 or bfloat16; ``logits``
    (tokens, experts) float32, -inf for experts a token may not take; W13
    (experts, 2*inner, hidden), gate rows first, and W2 (experts, hidden, inner)
    in X's type, or float8_e4m3fn with float32 scales S13 and S2 (one for each
    128 elements of a row, or for each 128 x 128 block).  ``renormalize``: the
    weights of a token's ``topk`` experts are normalised over those alone,
    otherwise over all of its experts.  ``workspace``, a contiguous tensor
    of :func:`gemm_nt_moe_workspace_bytes` bytes, is allocated if not given.
    """
    side = _elsewhere(stream)
    if side is not None:
        return _run_on(side, moe_few_tokens, X, logits, W13, W2, topk, S13, S2, renormalize, out, workspace, given=out)
    torch = _torch or _init_torch()
    xsh, lsh, s13h, s2h = X.shape, logits.shape, W13.shape, W2.shape
    if len(xsh) != 2 or len(lsh) != 2 or len(s13h) != 3 or len(s2h) != 3:
        raise ValueError(_MOE_SHAPES)
    tokens, hidden = xsh
    experts, inner = lsh[1], s2h[2]
    if lsh[0] != tokens or s13h != (experts, 2 * inner, hidden) or s2h != (experts, hidden, inner):
        raise ValueError(_MOE_SHAPES)
    xt = _one_of(X.dtype, _X16, "X")
    if W13.dtype != W2.dtype:
        raise TypeError("W13 and W2 must have the same type")
    wt = _one_of(W13.dtype, (X.dtype, torch.float8_e4m3fn), "W13 and W2")
    if logits.dtype != torch.float32:
        raise TypeError("logits must be float32")
    if (wt == 3) != (S13 is not None) or (S13 is None) != (S2 is None):
        raise ValueError("8-bit weights take S13 and S2, 16-bit weights none")
    s13 = s2 = None
    if S13 is not None:
        if S13.dim() != 3 or S2.dim() != 3 or S13.shape[0] != experts or S2.shape[0] != experts:
            raise ValueError("S13 and S2 need a leading expert dimension")
        s13, s2 = _scale128(S13, 2 * inner, hidden, "S13"), _scale128(S2, hidden, inner, "S2")
    index, device = _same_device(X, logits, W13, W2, S13, S2, out, workspace), X.device
    if out is None:
        out = torch.empty((tokens, hidden), dtype=X.dtype, device=device)
    elif tuple(out.shape) != (tokens, hidden) or out.dtype != X.dtype:
        raise ValueError("out must have X's shape and type")
    if workspace is None:
        # (what the library is going to refuse needs none)
        need = gemm_nt_moe_workspace_bytes(tokens, topk, inner) if 0 < topk <= experts and tokens <= 128 else 0
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=device)
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    t13, t2 = W13.stride(), W2.stride()
    gemm_nt_moe(X.data_ptr(), _pitch(xsh, X.stride(), "X"), logits.data_ptr(), _pitch(lsh, logits.stride(), "logits"),
                W13.data_ptr(), _pitch(s13h, t13, "W13"), t13[0], s13, W2.data_ptr(), _pitch(s2h, t2, "W2"), t2[0], s2,
                out.data_ptr(), _pitch(xsh, out.stride(), "out"), xt, wt, tokens, experts, topk, hidden, inner,
                renormalize, workspace.data_ptr(), workspace.nbytes, _stream_of(index))
    return out
