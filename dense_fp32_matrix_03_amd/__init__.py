"""Python binding of libsgemm: single-precision C = A x B on MI355X (gfx950).

Argument marshalling only.  Every function here forwards to the entry point
of the same name in libsgemm.so (declared in include/sgemm.h); all arithmetic
runs in the library's HIP kernels.  There is no CPU fallback: if the library
is missing, every call raises.

Matrices may be given as torch tensors on the GPU (their data pointer is
passed) or as plain integer device addresses.  ``stream`` may be a
torch.cuda.Stream, an integer hipStream_t, or None for torch's current stream
on the current device.
"""
from __future__ import annotations

import ctypes
import os
import re

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libsgemm.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "sgemm.h")
MXFP4_HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "sgemm_mxfp4.h")
ROUTE_HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "sgemm_route.h")
INT8_HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "sgemm_int8.h")


def _header_constants(path: str = HEADER_PATH) -> dict:
    out = {}
    with open(path) as f:
        for m in re.finditer(r"#define\s+(SGEMM_\w+)\s+\(?(-?\d+)\)?", f.read()):
            out[m.group(1)] = int(m.group(2))
    return out


_C = _header_constants()
SGEMM_OK = _C["SGEMM_OK"]
VARIANTS = {k[len("SGEMM_VARIANT_"):].lower(): v for k, v in _C.items()
            if k.startswith("SGEMM_VARIANT_")}
NUM_VARIANTS = _C["SGEMM_NUM_VARIANTS"]
# Element types of operands: "f32", "bf16", "mxfp4", "int8".
TYPES = {k[len("SGEMM_TYPE_"):].lower(): v for path in (MXFP4_HEADER_PATH, INT8_HEADER_PATH)
         for k, v in _header_constants(path).items() if k.startswith("SGEMM_TYPE_")}
# How sgemm_route makes scores of logits: "softmax", "sigmoid".
SCORES = {k[len("SGEMM_SCORE_"):].lower(): v
          for k, v in _header_constants(ROUTE_HEADER_PATH).items() if k.startswith("SGEMM_SCORE_")}


class SgemmError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {sgemm_status_string(status)} ({status})")


_lib = None


def load_library(path: str = LIB_PATH):
    """Load libsgemm.so and declare its signatures (raises if it is missing)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is not built; run `python -m dense_fp32_matrix_03_amd.build` "
            "(there is no fallback implementation)")
    lib = ctypes.CDLL(path)
    i64, vp, ci = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
    gemm_args = [i64, i64, i64, vp, i64, vp, i64, vp, i64, vp]
    lib.sgemm_create.argtypes = []
    lib.sgemm_create.restype = ci
    lib.sgemm_destroy.argtypes = []
    lib.sgemm_destroy.restype = ci
    lib.sgemm_run.argtypes = gemm_args
    lib.sgemm_run.restype = ci
    lib.sgemm_run_variant.argtypes = [ci] + gemm_args
    lib.sgemm_run_variant.restype = ci
    f32 = ctypes.c_float
    lib.sgemm_run_ex.argtypes = [ci, ci, i64, i64, i64, f32, vp, i64, vp, i64, f32, vp, i64, vp]
    lib.sgemm_run_ex.restype = ci
    lib.sgemm_run_strided_batched.argtypes = [ci, ci, i64, i64, i64, f32, vp, i64, i64, vp, i64,
                                              i64, f32, vp, i64, i64, i64, vp]
    lib.sgemm_run_strided_batched.restype = ci
    lib.sgemm_bf16x3_workspace_size.argtypes = [i64, i64, i64]
    lib.sgemm_bf16x3_workspace_size.restype = i64
    lib.sgemm_run_bf16x3.argtypes = gemm_args[:-1] + [vp, i64, vp]
    lib.sgemm_run_bf16x3.restype = ci
    lib.sgemm_run_bf16x3_ex.argtypes = [ci, ci, i64, i64, i64, f32, vp, i64, vp, i64, f32, vp,
                                        i64, vp, i64, vp]
    lib.sgemm_run_bf16x3_ex.restype = ci
    lib.sgemm_run_bf16x3_ex_noalloc.argtypes = [ci, ci, i64, i64, i64, f32, vp, i64, vp, i64,
                                                f32, vp, i64, vp]
    lib.sgemm_run_bf16x3_ex_noalloc.restype = ci
    lib.sgemm_run_grouped.argtypes = [ci, i64, i64, i64, i64, f32, vp, i64, vp, i64, i64, f32, vp,
                                      i64, vp, vp]
    lib.sgemm_run_grouped.restype = ci
    lib.sgemm_run_grouped_k.argtypes = [i64, i64, i64, i64, f32, vp, i64, vp, i64, f32, vp, i64,
                                        i64, vp, vp]
    lib.sgemm_run_grouped_k.restype = ci
    for size in (lib.sgemm_mxfp4_codes_size, lib.sgemm_mxfp4_scales_size):
        size.argtypes = [i64, i64]
        size.restype = i64
    lib.sgemm_mxfp4_workspace_size.argtypes = [ci, i64, i64]
    lib.sgemm_mxfp4_workspace_size.restype = i64
    lib.sgemm_mxfp4_quantize.argtypes = [ci, i64, i64, ci, vp, i64, vp, vp, i64, vp]
    lib.sgemm_mxfp4_quantize.restype = ci
    lib.sgemm_mxfp4_dequantize.argtypes = [ci, i64, i64, vp, vp, i64, ci, vp, i64, vp]
    lib.sgemm_mxfp4_dequantize.restype = ci
    mxfp4_args = [i64, i64, i64, f32, ci, vp, i64, vp, vp, vp, i64, f32, ci, vp, i64]
    lib.sgemm_run_mxfp4.argtypes = mxfp4_args + [vp, i64, vp]
    lib.sgemm_run_mxfp4.restype = ci
    lib.sgemm_run_mxfp4_grouped.argtypes = [i64] + mxfp4_args + [vp, vp, i64, vp]
    lib.sgemm_run_mxfp4_grouped.restype = ci
    lib.sgemm_int8_codes_size.argtypes = [i64, i64]
    lib.sgemm_int8_codes_size.restype = i64
    lib.sgemm_int8_workspace_size.argtypes = [ci, i64, i64]
    lib.sgemm_int8_workspace_size.restype = i64
    lib.sgemm_int8_quantize.argtypes = [ci, i64, i64, ci, vp, i64, vp, i64, vp, vp]
    lib.sgemm_int8_quantize.restype = ci
    int8_args = [i64, i64, i64, f32, ci, vp, i64, vp, vp, i64, vp, f32, ci, vp, i64]
    lib.sgemm_run_int8.argtypes = int8_args + [vp, i64, vp]
    lib.sgemm_run_int8.restype = ci
    lib.sgemm_run_int8_grouped.argtypes = [i64] + int8_args + [vp, vp, i64, vp]
    lib.sgemm_run_int8_grouped.restype = ci
    route_args = [i64, i64, i64, ci, ci, vp, i64]
    lib.sgemm_route.argtypes = route_args + [vp, i64, i64, i64, ci, f32, vp, vp, vp]
    lib.sgemm_route.restype = ci
    lib.sgemm_route_backward.argtypes = route_args + [ci, f32, vp, vp, vp, i64, vp]
    lib.sgemm_route_backward.restype = ci
    lib.sgemm_route_plan_workspace_size.argtypes = [i64, i64]
    lib.sgemm_route_plan_workspace_size.restype = i64
    lib.sgemm_route_plan.argtypes = [i64, i64, i64, vp, vp, vp, vp, vp, i64, vp]
    lib.sgemm_route_plan.restype = ci
    rows_args = [i64, i64, i64, i64, ci, vp, i64]
    lib.sgemm_rows_gather.argtypes = rows_args + [vp, vp, vp, i64, vp]
    lib.sgemm_rows_gather.restype = ci
    lib.sgemm_rows_combine.argtypes = rows_args + [vp, vp, vp, i64, vp]
    lib.sgemm_rows_combine.restype = ci
    lib.sgemm_rows_combine_backward.argtypes = rows_args + [vp, i64, vp, vp, vp, i64, vp, vp]
    lib.sgemm_rows_combine_backward.restype = ci
    lib.sgemm_orthogonalize_workspace_size.argtypes = [i64, i64, i64]
    lib.sgemm_orthogonalize_workspace_size.restype = i64
    lib.sgemm_orthogonalize.argtypes = [i64, i64, i64, i64, i64, ctypes.POINTER(f32), f32, f32, ci,
                                        vp, i64, i64, ci, vp, i64, i64, vp, i64, vp]
    lib.sgemm_orthogonalize.restype = ci
    lib.vector_add.argtypes = [i64, vp, vp, vp, vp]
    lib.vector_add.restype = ci
    lib.sgemm_mfma_ceiling.argtypes = [ci, ci, vp, i64, ctypes.POINTER(ctypes.c_double), vp]
    lib.sgemm_mfma_ceiling.restype = ci
    lib.sgemm_phase_times.argtypes = gemm_args[:-1] + [vp, i64, ctypes.POINTER(i64), vp]
    lib.sgemm_phase_times.restype = ci
    pi = ctypes.POINTER(ci)
    lib.sgemm_tile_choice.argtypes = [i64, i64, i64, i64, ci, pi, pi, pi, pi]
    lib.sgemm_tile_choice.restype = ci
    lib.sgemm_mfma_probe.argtypes = [ci, vp, vp, vp, vp]
    lib.sgemm_mfma_probe.restype = ci
    lib.sgemm_status_string.argtypes = [ci]
    lib.sgemm_status_string.restype = ctypes.c_char_p
    lib.sgemm_variant_name.argtypes = [ci]
    lib.sgemm_variant_name.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _ptr(x):
    if x is None or isinstance(x, int):
        return x
    try:
        data_ptr = x.data_ptr
    except AttributeError:
        raise TypeError(f"cannot take a device pointer from {type(x).__name__}") from None
    try:
        on_gpu = x.is_cuda
    except AttributeError:
        on_gpu = getattr(x, "device", None) is None or x.device.type == "cuda"
    if not on_gpu:
        raise ValueError("tensor must live on the GPU")
    return data_ptr()


_current_stream = None


def _find_current_stream():
    """A function that returns torch's current stream on the current device as
    an integer.  Building a torch.cuda.Stream object for each call takes 2.8
    us, as long as a launch; the handle alone takes 0.2."""
    import torch
    torch.cuda.current_stream()  # initialises torch's side
    try:
        raw, device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
        raw(device())
    except AttributeError:
        return lambda: torch.cuda.current_stream().cuda_stream
    return lambda: raw(device())


def _stream(s):
    if s is None:
        global _current_stream
        if _current_stream is None:
            _current_stream = _find_current_stream()
        return _current_stream()
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _type(t) -> int:
    return TYPES[t] if isinstance(t, str) else int(t)


def _score(s) -> int:
    return SCORES[s] if isinstance(s, str) else int(s)


def _offsets(x, groups=0):
    """_ptr of group offsets, which the kernels read as groups + 1 64-bit integers."""
    if hasattr(x, "dtype"):
        if x.element_size() != 8 or x.is_floating_point() or x.is_complex():
            raise TypeError("offsets must be int64")
        if not x.is_contiguous():
            raise ValueError("offsets must be contiguous")
        if groups > 0 and x.numel() <= groups:
            raise ValueError(f"offsets must hold groups + 1 = {groups + 1} values, not {x.numel()}")
    return _ptr(x)


_dtypes = {}


def _typed(x, name, dtype, size=0):
    """_ptr of `size` contiguous 32-bit values, of which the kernels know only the address."""
    if x is None or isinstance(x, int):
        return x
    want = _dtypes.get(dtype)
    if want is None:
        import torch
        want = _dtypes[dtype] = getattr(torch, dtype)
    try:  # all at once: 0.2 us where the checks below take 0.4
        if x.dtype is want and x.is_cuda and x.numel() >= size and x.is_contiguous():
            return x.data_ptr()
    except AttributeError:
        pass
    if getattr(x, "dtype", want) is not want:
        raise TypeError(f"{name} must be {dtype}")
    if hasattr(x, "numel"):
        if not x.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if x.numel() < size:
            raise ValueError(f"{name} must hold {size} values, not {x.numel()}")
    return _ptr(x)


def _size(fn: str, *args) -> int:
    r = getattr(load_library(), fn)(*args)
    if r < 0:
        raise SgemmError(fn, int(r))
    return int(r)


def _check(fn: str, status: int) -> None:
    if status != SGEMM_OK:
        raise SgemmError(fn, status)


def sgemm_create() -> None:
    _check("sgemm_create", load_library().sgemm_create())


def sgemm_destroy() -> None:
    _check("sgemm_destroy", load_library().sgemm_destroy())


def sgemm_run(M, N, K, A, lda, B, ldb, C, ldc, stream=None) -> None:
    """C = A x B (row-major, leading dimensions lda, ldb, ldc) on `stream`."""
    _check("sgemm_run", load_library().sgemm_run(
        M, N, K, _ptr(A), lda, _ptr(B), ldb, _ptr(C), ldc, _stream(stream)))


def sgemm_run_variant(variant, M, N, K, A, lda, B, ldb, C, ldc, stream=None) -> None:
    """sgemm_run computed by kernel `variant` (an int or a VARIANTS key)."""
    v = VARIANTS[variant] if isinstance(variant, str) else int(variant)
    _check("sgemm_run_variant", load_library().sgemm_run_variant(
        v, M, N, K, _ptr(A), lda, _ptr(B), ldb, _ptr(C), ldc, _stream(stream)))


def sgemm_run_ex(transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
                 stream=None) -> None:
    """C = alpha op(A) op(B) + beta C (op = transpose when the flag is set)."""
    _check("sgemm_run_ex", load_library().sgemm_run_ex(
        int(transA), int(transB), M, N, K, float(alpha), _ptr(A), lda, _ptr(B), ldb,
        float(beta), _ptr(C), ldc, _stream(stream)))


def sgemm_tile_choice(M, N, K, batch=1, cus=256) -> tuple:
    """(bm, bn, bk, ksets) that sgemm_run and the general form choose for
    `batch` products of M x N x K on `cus` compute units (host logic only)."""
    out = [ctypes.c_int() for _ in range(4)]
    _check("sgemm_tile_choice", load_library().sgemm_tile_choice(
        M, N, K, batch, cus, *(ctypes.byref(o) for o in out)))
    return tuple(o.value for o in out)


def sgemm_run_strided_batched(transA, transB, M, N, K, alpha, A, lda, strideA, B, ldb,
                              strideB, beta, C, ldc, strideC, batch, stream=None) -> None:
    """`batch` general products, operands `stride*` floats apart."""
    _check("sgemm_run_strided_batched", load_library().sgemm_run_strided_batched(
        int(transA), int(transB), M, N, K, float(alpha), _ptr(A), lda, strideA, _ptr(B), ldb,
        strideB, float(beta), _ptr(C), ldc, strideC, batch, _stream(stream)))


def sgemm_bf16x3_workspace_size(M, N, K) -> int:
    """Workspace bytes sgemm_run_bf16x3 needs (include/sgemm_bf16x3.h)."""
    r = load_library().sgemm_bf16x3_workspace_size(M, N, K)
    if r < 0:
        raise SgemmError("sgemm_bf16x3_workspace_size", int(r))
    return int(r)


def sgemm_run_bf16x3(M, N, K, A, lda, B, ldb, C, ldc, workspace, workspace_bytes,
                     stream=None) -> None:
    """C = A x B on the bfloat16 matrix cores (three-piece split)."""
    _check("sgemm_run_bf16x3", load_library().sgemm_run_bf16x3(
        M, N, K, _ptr(A), lda, _ptr(B), ldb, _ptr(C), ldc, _ptr(workspace), workspace_bytes,
        _stream(stream)))


def sgemm_run_bf16x3_ex(transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
                        workspace, workspace_bytes, stream=None) -> None:
    """C = alpha op(A) op(B) + beta C on the bfloat16 matrix cores."""
    _check("sgemm_run_bf16x3_ex", load_library().sgemm_run_bf16x3_ex(
        int(transA), int(transB), M, N, K, float(alpha), _ptr(A), lda, _ptr(B), ldb,
        float(beta), _ptr(C), ldc, _ptr(workspace), workspace_bytes, _stream(stream)))


def sgemm_run_bf16x3_ex_noalloc(transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
                                stream=None) -> None:
    """sgemm_run_bf16x3_ex with the library-held split buffer (no workspace)."""
    _check("sgemm_run_bf16x3_ex_noalloc", load_library().sgemm_run_bf16x3_ex_noalloc(
        int(transA), int(transB), M, N, K, float(alpha), _ptr(A), lda, _ptr(B), ldb,
        float(beta), _ptr(C), ldc, _stream(stream)))


def sgemm_run_grouped(transB, groups, M, N, K, alpha, A, lda, B, ldb, strideB, beta, C, ldc,
                      offsets, stream=None) -> None:
    """C(r, :) = alpha A(r, :) op(B_g) + beta C(r, :) for the rows r of each
    group g (include/sgemm_grouped.h); offsets: groups + 1 int64 on the GPU."""
    _check("sgemm_run_grouped", load_library().sgemm_run_grouped(
        int(transB), groups, M, N, K, float(alpha), _ptr(A), lda, _ptr(B), ldb, strideB,
        float(beta), _ptr(C), ldc, _offsets(offsets, groups), _stream(stream)))


def sgemm_run_grouped_k(groups, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, strideC, offsets,
                        stream=None) -> None:
    """C_g = alpha A_g^T B_g + beta C_g over the rows of each group g: the
    gradient of sgemm_run_grouped's B (include/sgemm_grouped.h)."""
    _check("sgemm_run_grouped_k", load_library().sgemm_run_grouped_k(
        groups, M, N, K, float(alpha), _ptr(A), lda, _ptr(B), ldb, float(beta), _ptr(C), ldc,
        strideC, _offsets(offsets, groups), _stream(stream)))


def sgemm_mxfp4_codes_size(rows, K) -> int:
    """Bytes of the codes of a held rows x K matrix (include/sgemm_mxfp4.h)."""
    return _size("sgemm_mxfp4_codes_size", rows, K)


def sgemm_mxfp4_scales_size(rows, K) -> int:
    """Bytes of its scales, with lds = rows."""
    return _size("sgemm_mxfp4_scales_size", rows, K)


def sgemm_mxfp4_workspace_size(typeA, M, K) -> int:
    """Workspace bytes of a 4-bit product whose A has type `typeA`."""
    return _size("sgemm_mxfp4_workspace_size", _type(typeA), M, K)


def sgemm_mxfp4_quantize(trans, rows, K, type, X, ldx, codes, scales, lds, stream=None) -> None:
    """Cast X (rows x K, or with trans stored K x rows; type "f32" or "bf16")
    to microscaled 4-bit floats."""
    _check("sgemm_mxfp4_quantize", load_library().sgemm_mxfp4_quantize(
        int(trans), rows, K, _type(type), _ptr(X), ldx, _ptr(codes), _ptr(scales), lds,
        _stream(stream)))


def sgemm_mxfp4_dequantize(trans, rows, K, codes, scales, lds, type, X, ldx, stream=None) -> None:
    """The values of a held matrix, written to X as sgemm_mxfp4_quantize reads it."""
    _check("sgemm_mxfp4_dequantize", load_library().sgemm_mxfp4_dequantize(
        int(trans), rows, K, _ptr(codes), _ptr(scales), lds, _type(type), _ptr(X), ldx,
        _stream(stream)))


def sgemm_run_mxfp4(M, N, K, alpha, typeA, A, lda, scalesA, B, scalesB, ldsb, beta, typeC, C, ldc,
                    workspace=None, workspace_bytes=0, stream=None) -> None:
    """C = alpha A B^T + beta C with B (and, for typeA "mxfp4", A) held in
    microscaled 4-bit floats; an "f32" or "bf16" A is cast on the way."""
    _check("sgemm_run_mxfp4", load_library().sgemm_run_mxfp4(
        M, N, K, float(alpha), _type(typeA), _ptr(A), lda, _ptr(scalesA), _ptr(B), _ptr(scalesB),
        ldsb, float(beta), _type(typeC), _ptr(C), ldc, _ptr(workspace), workspace_bytes,
        _stream(stream)))


def sgemm_run_mxfp4_grouped(groups, M, N, K, alpha, typeA, A, lda, scalesA, B, scalesB, ldsb, beta,
                            typeC, C, ldc, offsets, workspace=None, workspace_bytes=0,
                            stream=None) -> None:
    """sgemm_run_mxfp4 for rows in groups, group g with rows g N .. of B."""
    _check("sgemm_run_mxfp4_grouped", load_library().sgemm_run_mxfp4_grouped(
        groups, M, N, K, float(alpha), _type(typeA), _ptr(A), lda, _ptr(scalesA), _ptr(B),
        _ptr(scalesB), ldsb, float(beta), _type(typeC), _ptr(C), ldc, _offsets(offsets, groups),
        _ptr(workspace), workspace_bytes, _stream(stream)))


def sgemm_int8_codes_size(rows, K) -> int:
    """Bytes of the codes of a held rows x K matrix, ldq = K padded to 128 (include/sgemm_int8.h)."""
    return _size("sgemm_int8_codes_size", rows, K)


def sgemm_int8_workspace_size(typeA, M, K) -> int:
    """Workspace bytes of an 8-bit product whose A has type `typeA`."""
    return _size("sgemm_int8_workspace_size", _type(typeA), M, K)


def sgemm_int8_quantize(trans, rows, K, type, X, ldx, codes, ldq, scales, stream=None) -> None:
    """Cast X (rows x K, or with trans stored K x rows; type "f32" or "bf16") to 8-bit integers
    with a scale for each row."""
    _check("sgemm_int8_quantize", load_library().sgemm_int8_quantize(
        int(trans), rows, K, _type(type), _ptr(X), ldx, _ptr(codes), ldq,
        _typed(scales, "scales", "float32", rows), _stream(stream)))


def _scales_a(typeA, scales, M):
    """A's scales, which are read only where A is held."""
    return _typed(scales, "scalesA", "float32", M if _type(typeA) == TYPES["int8"] else 0)


def sgemm_run_int8(M, N, K, alpha, typeA, A, lda, scalesA, B, ldb, scalesB, beta, typeC, C, ldc,
                   workspace=None, workspace_bytes=0, stream=None) -> None:
    """C = alpha A B^T + beta C with B (and, for typeA "int8", A) held in 8-bit integers; an "f32"
    or "bf16" A is cast on the way."""
    _check("sgemm_run_int8", load_library().sgemm_run_int8(
        M, N, K, float(alpha), _type(typeA), _ptr(A), lda, _scales_a(typeA, scalesA, M), _ptr(B),
        ldb, _typed(scalesB, "scalesB", "float32", N), float(beta), _type(typeC), _ptr(C), ldc,
        _ptr(workspace), workspace_bytes, _stream(stream)))


def sgemm_run_int8_grouped(groups, M, N, K, alpha, typeA, A, lda, scalesA, B, ldb, scalesB, beta,
                           typeC, C, ldc, offsets, workspace=None, workspace_bytes=0,
                           stream=None) -> None:
    """sgemm_run_int8 for rows in groups, group g with rows g N .. of B."""
    _check("sgemm_run_int8_grouped", load_library().sgemm_run_int8_grouped(
        groups, M, N, K, float(alpha), _type(typeA), _ptr(A), lda, _scales_a(typeA, scalesA, M),
        _ptr(B), ldb, _typed(scalesB, "scalesB", "float32", groups * N), float(beta), _type(typeC),
        _ptr(C), ldc, _offsets(offsets, groups), _ptr(workspace), workspace_bytes,
        _stream(stream)))


def sgemm_route(tokens, experts, topk, score, type, logits, ldl, bias, groups, topk_groups,
                group_top, renormalize, scale, picks, weights, stream=None) -> None:
    """The topk experts of each token and their weights, from logits (include/sgemm_route.h);
    score: "softmax" or "sigmoid", picks int32, weights float32, tokens x topk."""
    _check("sgemm_route", load_library().sgemm_route(
        tokens, experts, topk, _score(score), _type(type), _ptr(logits), ldl,
        _typed(bias, "bias", "float32", experts), groups, topk_groups, group_top,
        int(renormalize), float(scale), _typed(picks, "picks", "int32", tokens * topk),
        _typed(weights, "weights", "float32", tokens * topk), _stream(stream)))


def sgemm_route_backward(tokens, experts, topk, score, type, logits, ldl, renormalize, scale, picks,
                         dweights, dlogits, ldd, stream=None) -> None:
    """The gradient of sgemm_route's weights with respect to its logits."""
    _check("sgemm_route_backward", load_library().sgemm_route_backward(
        tokens, experts, topk, _score(score), _type(type), _ptr(logits), ldl, int(renormalize),
        float(scale), _typed(picks, "picks", "int32", tokens * topk),
        _typed(dweights, "dweights", "float32", tokens * topk), _ptr(dlogits), ldd,
        _stream(stream)))


def sgemm_route_plan_workspace_size(pairs, groups) -> int:
    """Workspace bytes of sgemm_route_plan."""
    return _size("sgemm_route_plan_workspace_size", pairs, groups)


def sgemm_route_plan(pairs, first, groups, picks, offsets, sources, places, workspace=None,
                     workspace_bytes=0, stream=None) -> None:
    """Sort pairs (token, pick) by expert: the groups' offsets (int64), the pair of each row and
    the row of each pair (int32)."""
    _check("sgemm_route_plan", load_library().sgemm_route_plan(
        pairs, first, groups, _typed(picks, "picks", "int32", pairs), _offsets(offsets, groups),
        _typed(sources, "sources", "int32", pairs), _typed(places, "places", "int32", pairs),
        _ptr(workspace), workspace_bytes, _stream(stream)))


def sgemm_rows_gather(rows, pairs, topk, N, type, X, ldx, sources, weights, Y, ldy,
                      stream=None) -> None:
    """Y(r, :) = weights[sources[r]] X(sources[r] / topk, :), weights None for ones."""
    _check("sgemm_rows_gather", load_library().sgemm_rows_gather(
        rows, pairs, topk, N, _type(type), _ptr(X), ldx, _typed(sources, "sources", "int32", rows),
        _typed(weights, "weights", "float32", pairs), _ptr(Y), ldy, _stream(stream)))


def sgemm_rows_combine(tokens, topk, rows, N, type, X, ldx, places, weights, Y, ldy,
                       stream=None) -> None:
    """Y(t, :) = sum_j weights[t, j] X(places[t, j], :), weights None for ones."""
    _check("sgemm_rows_combine", load_library().sgemm_rows_combine(
        tokens, topk, rows, N, _type(type), _ptr(X), ldx,
        _typed(places, "places", "int32", tokens * topk),
        _typed(weights, "weights", "float32", tokens * topk), _ptr(Y), ldy, _stream(stream)))


def sgemm_rows_combine_backward(tokens, topk, rows, N, type, X, ldx, dY, lddy, places, weights, dX,
                                lddx, dweights, stream=None) -> None:
    """The gradients dX and dweights (either may be None) of sgemm_rows_combine."""
    pairs = tokens * topk
    _check("sgemm_rows_combine_backward", load_library().sgemm_rows_combine_backward(
        tokens, topk, rows, N, _type(type), _ptr(X), ldx, _ptr(dY), lddy,
        _typed(places, "places", "int32", pairs), _typed(weights, "weights", "float32", pairs),
        _ptr(dX), lddx, _typed(dweights, "dweights", "float32", pairs), _stream(stream)))


def sgemm_orthogonalize_workspace_size(batch, M, N) -> int:
    """Workspace bytes of sgemm_orthogonalize."""
    return _size("sgemm_orthogonalize_workspace_size", batch, M, N)


def sgemm_orthogonalize(batch, M, N, steps, coefficients, eps, alpha, typeX, X, ldx, strideX, typeY,
                        Y, ldy, strideY, workspace=None, workspace_bytes=0, stream=None) -> None:
    """Y = alpha times the Newton-Schulz iterate of each X / (|X| + eps)
    (include/sgemm_orthogonalize.h); coefficients: a, b, c for all steps alike, or 3 * steps."""
    n = len(coefficients)
    if n not in (3, 3 * steps):
        raise ValueError(f"coefficients must hold 3 or 3 * steps = {3 * steps} values, not {n}")
    _check("sgemm_orthogonalize", load_library().sgemm_orthogonalize(
        batch, M, N, steps, n // 3, (ctypes.c_float * n)(*coefficients), float(eps), float(alpha),
        _type(typeX), _ptr(X), ldx, strideX, _type(typeY), _ptr(Y), ldy, strideY, _ptr(workspace),
        workspace_bytes, _stream(stream)))


def vector_add(n, A, B, C, stream=None) -> None:
    """C[i] = A[i] + B[i] for i < n (include/vector_add.h)."""
    _check("vector_add", load_library().vector_add(n, _ptr(A), _ptr(B), _ptr(C),
                                                   _stream(stream)))


def sgemm_mfma_ceiling(which, iters, out, out_len, stream=None) -> float:
    """Launch the register-only matrix-core loop; return its flop count."""
    flops = ctypes.c_double(0.0)
    _check("sgemm_mfma_ceiling", load_library().sgemm_mfma_ceiling(
        int(which), int(iters), _ptr(out), int(out_len), ctypes.byref(flops), _stream(stream)))
    return flops.value


def sgemm_phase_times(M, N, K, A, lda, B, ldb, C, ldc, times, times_len, stream=None) -> int:
    """sgemm_run with per-work-group phase timestamps in `times` (8 uint64
    per work-group; times=None only queries); returns the work-group count."""
    wgs = ctypes.c_int64(0)
    _check("sgemm_phase_times", load_library().sgemm_phase_times(
        M, N, K, _ptr(A), lda, _ptr(B), ldb, _ptr(C), ldc, _ptr(times), int(times_len),
        ctypes.byref(wgs), _stream(stream)))
    return wgs.value


def sgemm_mfma_probe(which, A, B, C, stream=None) -> None:
    _check("sgemm_mfma_probe", load_library().sgemm_mfma_probe(
        int(which), _ptr(A), _ptr(B), _ptr(C), _stream(stream)))


def sgemm_status_string(status: int) -> str:
    return load_library().sgemm_status_string(int(status)).decode()


def sgemm_variant_name(variant: int):
    s = load_library().sgemm_variant_name(int(variant))
    return s.decode() if s is not None else None


def matmul(A, B, out=None, variant=None, stream=None):
    """C = A @ B for 2-D float32 torch tensors on the GPU (row-major, unit
    column stride; row strides become the leading dimensions).  Allocates
    `out` with torch when it is not given."""
    import torch
    if A.dtype != torch.float32 or B.dtype != torch.float32:
        raise TypeError("A and B must be float32")
    if A.dim() != 2 or B.dim() != 2 or A.shape[1] != B.shape[0]:
        raise ValueError(f"shapes {tuple(A.shape)} x {tuple(B.shape)} do not chain")
    M, K = A.shape
    N = B.shape[1]
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=A.device)
    for name, t in (("A", A), ("B", B), ("out", out)):
        if t.dim() == 2 and t.shape[0] > 0 and t.shape[1] > 1 and t.stride(1) != 1:
            raise ValueError(f"{name} must have unit column stride")
    lda = max(A.stride(0), 1) if M > 0 else max(K, 1)
    ldb = max(B.stride(0), 1) if K > 0 else max(N, 1)
    ldc = max(out.stride(0), 1) if M > 0 else max(N, 1)
    if variant is None:
        sgemm_run(M, N, K, A, lda, B, ldb, out, ldc, stream)
    else:
        sgemm_run_variant(variant, M, N, K, A, lda, B, ldb, out, ldc, stream)
    return out
