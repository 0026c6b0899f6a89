"""Python binding of libgemm_f32.so (argument marshalling only).

The functions mirror the C entry points of ``include/gemm_f32.h`` one to one;
every step of the product runs in the library's HIP kernels.  torch provides
device memory and streams: matrix arguments may be torch CUDA tensors (their
``data_ptr()``, which includes any storage offset) or raw device addresses.

torch is imported before the library is loaded so that both use torch's HIP
runtime.  There is no fallback: if the library is missing and cannot be
built, or a call returns a nonzero status, an exception is raised.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading

import torch  # noqa: F401  (must precede loading the HIP library)

_PKG = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_PKG, "libgemm_f32.so")

_i64 = ctypes.c_int64
_vp = ctypes.c_void_p
_lib = None
_lock = threading.Lock()

OK = 0
VARIANTS = {"naive": 0, "tiled": 1, "regblock": 2, "mfma": 3}
OPS = {"N": 0, "T": 1, 0: 0, 1: 1}
DIAGNOSTIC_BASE = 16


class Epilogue(ctypes.Structure):
    """gemm_epilogue of gemm_f32.h."""
    _fields_ = [("c_type", ctypes.c_int), ("activation", ctypes.c_int), ("gradient", ctypes.c_int),
                ("bias_type", ctypes.c_int), ("bias", _vp), ("residual", _vp), ("ld_residual", _i64),
                ("preact", _vp), ("ld_preact", _i64), ("bias_grad", _vp)]


class GemmError(RuntimeError):
    """A nonzero status returned by the library."""

    def __init__(self, status: int, message: str):
        super().__init__(f"gemm_f32 status {status}: {message}")
        self.status = status


def load_library():
    """Loads libgemm_f32.so, building it only if no built library exists."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(library_path):
            from . import build as _build
            _build.build()
        lib = ctypes.CDLL(library_path)
        sig = [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp]
        lib.gemm_f32.argtypes = sig
        lib.gemm_f32.restype = ctypes.c_int
        lib.gemm_f32_variant.argtypes = [ctypes.c_int] + sig
        lib.gemm_f32_variant.restype = ctypes.c_int
        lib.gemm_f32_op.argtypes = [ctypes.c_int, ctypes.c_int] + sig
        lib.gemm_f32_op.restype = ctypes.c_int
        lib.gemm_f32_num_variants.argtypes = []
        lib.gemm_f32_num_variants.restype = ctypes.c_int
        lib.gemm_f32_num_diagnostic_variants.argtypes = []
        lib.gemm_f32_num_diagnostic_variants.restype = ctypes.c_int
        lib.gemm_f32_variant_name.argtypes = [ctypes.c_int]
        lib.gemm_f32_variant_name.restype = ctypes.c_char_p
        lib.gemm_f32_status_string.argtypes = [ctypes.c_int]
        lib.gemm_f32_status_string.restype = ctypes.c_char_p
        lib.gemm_f32_default_variant.argtypes = [_i64, _i64, _i64]
        lib.gemm_f32_default_variant.restype = ctypes.c_int
        tsig = [_i64, _i64, _vp, _i64, _vp, _i64, _vp]
        lib.transpose_f32.argtypes = tsig
        lib.transpose_f32.restype = ctypes.c_int
        lib.transpose_f32_variant.argtypes = [ctypes.c_int] + tsig
        lib.transpose_f32_variant.restype = ctypes.c_int
        lib.transpose_f32_num_variants.argtypes = []
        lib.transpose_f32_num_variants.restype = ctypes.c_int
        lib.transpose_f32_variant_name.argtypes = [ctypes.c_int]
        lib.transpose_f32_variant_name.restype = ctypes.c_char_p
        lib.transpose_f32_default_variant.argtypes = [_i64, _i64, _i64, _i64]
        lib.transpose_f32_default_variant.restype = ctypes.c_int
        lib.reduce_sum_f32_workspace_size.argtypes = [ctypes.c_int, _i64]
        lib.reduce_sum_f32_workspace_size.restype = _i64
        rsig = [_i64, _vp, _vp, _vp, _i64, _vp]
        lib.reduce_sum_f32.argtypes = rsig
        lib.reduce_sum_f32.restype = ctypes.c_int
        lib.reduce_sum_f32_variant.argtypes = [ctypes.c_int] + rsig
        lib.reduce_sum_f32_variant.restype = ctypes.c_int
        lib.gemm_f32_valu_probe.argtypes = [ctypes.c_int, _i64, ctypes.c_int, _vp, _vp, _vp]
        lib.gemm_f32_valu_probe.restype = ctypes.c_int
        lib.gemm_f32_lds_probe.argtypes = [ctypes.c_int, _vp, ctypes.c_int, _vp, _vp]
        lib.gemm_f32_lds_probe.restype = ctypes.c_int
        lib.gemm_f32_copy_probe.argtypes = [ctypes.c_int, _i64, ctypes.c_int, _vp, _vp, _vp, _vp]
        lib.gemm_f32_copy_probe.restype = ctypes.c_int
        lib.gemm_f32_ksplit_timeline.argtypes = sig[:-1] + [_vp, _i64, _vp]
        lib.gemm_f32_ksplit_timeline.restype = ctypes.c_int
        lib.reduce_sum_f32_variant_noalloc.argtypes = [ctypes.c_int, _i64, _vp, _vp, _vp]
        lib.reduce_sum_f32_variant_noalloc.restype = ctypes.c_int
        lib.reduce_sum_f32_num_variants.argtypes = []
        lib.reduce_sum_f32_num_variants.restype = ctypes.c_int
        lib.reduce_sum_f32_variant_name.argtypes = [ctypes.c_int]
        lib.reduce_sum_f32_variant_name.restype = ctypes.c_char_p
        msig = [ctypes.c_int] + sig
        lib.gemm_mixed.argtypes = msig
        lib.gemm_mixed.restype = ctypes.c_int
        lib.gemm_mixed_variant.argtypes = [ctypes.c_int] + msig
        lib.gemm_mixed_variant.restype = ctypes.c_int
        lib.gemm_mixed_op.argtypes = [ctypes.c_int, ctypes.c_int] + msig
        lib.gemm_mixed_op.restype = ctypes.c_int
        lib.gemm_mixed_num_variants.argtypes = []
        lib.gemm_mixed_num_variants.restype = ctypes.c_int
        lib.gemm_mixed_default_variant.argtypes = [_i64, _i64, _i64]
        lib.gemm_mixed_default_variant.restype = ctypes.c_int
        lib.gemm_mixed_variant_name.argtypes = [ctypes.c_int]
        lib.gemm_mixed_variant_name.restype = ctypes.c_char_p
        esig = [ctypes.c_int] * 3 + [_i64] * 3 + [_vp, _i64, _vp, _i64]
        ep = ctypes.POINTER(Epilogue)
        lib.gemm_mixed_epilogue_workspace_size.argtypes = esig + [ep]
        lib.gemm_mixed_epilogue_workspace_size.restype = _i64
        lib.gemm_mixed_epilogue.argtypes = esig + [_vp, _i64, ep, _vp, _i64, _vp]
        lib.gemm_mixed_epilogue.restype = ctypes.c_int
        lib.activation_grad_workspace_size.argtypes = [_i64, _i64]
        lib.activation_grad_workspace_size.restype = _i64
        lib.activation_grad.argtypes = [ctypes.c_int, ctypes.c_int, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp,
                                        _vp, _i64, _vp]
        lib.activation_grad.restype = ctypes.c_int
        lib.layer_norm.argtypes = [ctypes.c_int, _i64, _i64, _vp, _i64, ctypes.c_int, _vp, _vp, ctypes.c_float, _vp,
                                   _i64, _vp, _vp, _vp]
        lib.layer_norm.restype = ctypes.c_int
        lib.layer_norm_backward_workspace_size.argtypes = [ctypes.c_int, _i64, _i64]
        lib.layer_norm_backward_workspace_size.restype = _i64
        lib.layer_norm_backward.argtypes = [ctypes.c_int, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _vp, ctypes.c_int,
                                            _vp, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _vp]
        lib.layer_norm_backward.restype = ctypes.c_int
        lib.newton_schulz_workspace_size.argtypes = [ctypes.c_int, _i64, _i64, _i64]
        lib.newton_schulz_workspace_size.restype = _i64
        lib.newton_schulz.argtypes = [ctypes.c_int, _i64, _i64, _i64, _vp, _i64, _i64, ctypes.c_int] + \
            [ctypes.c_float] * 4 + [_vp, _i64, _i64, _vp, _i64, _vp]
        lib.newton_schulz.restype = ctypes.c_int
        _lib = lib
        return lib


def _addr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, torch.Tensor):
        if x.numel() and not x.is_cuda:
            raise TypeError("matrix tensors must live on the GPU")
        return x.data_ptr()
    return int(x)


def _stream(stream) -> int | None:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream if torch.cuda.is_available() else None
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _check(status: int) -> None:
    if status != OK:
        raise GemmError(status, gemm_f32_status_string(status))


def gemm_f32(M, N, K, A, lda, B, ldb, C, ldc, stream=None) -> None:
    """C = A x B on the library's default kernel; see gemm_f32.h."""
    lib = load_library()
    _check(lib.gemm_f32(M, N, K, _addr(A), lda, _addr(B), ldb, _addr(C), ldc, _stream(stream)))


def gemm_f32_variant(variant, M, N, K, A, lda, B, ldb, C, ldc, stream=None) -> None:
    """C = A x B on a chosen rung (0..3) or diagnostic variant (16..)."""
    lib = load_library()
    if isinstance(variant, str):
        variant = VARIANTS[variant]
    _check(lib.gemm_f32_variant(int(variant), M, N, K, _addr(A), lda, _addr(B), ldb,
                                _addr(C), ldc, _stream(stream)))


def gemm_f32_op(op_a, op_b, M, N, K, A, lda, B, ldb, C, ldc, stream=None) -> None:
    """C = op(A) x op(B), op 'N' (as stored) or 'T' (stored transposed)."""
    lib = load_library()
    oa = OPS.get(op_a, op_a) if not isinstance(op_a, int) else op_a
    ob = OPS.get(op_b, op_b) if not isinstance(op_b, int) else op_b
    _check(lib.gemm_f32_op(int(oa), int(ob), M, N, K, _addr(A), lda, _addr(B), ldb,
                           _addr(C), ldc, _stream(stream)))


def gemm_f32_num_variants() -> int:
    return load_library().gemm_f32_num_variants()


def gemm_f32_num_diagnostic_variants() -> int:
    return load_library().gemm_f32_num_diagnostic_variants()


def gemm_f32_default_variant(M, N, K) -> int:
    """The diagnostic variant whose configuration gemm_f32 runs for M x N x K
    (-1 for invalid sizes); no device needed."""
    return int(load_library().gemm_f32_default_variant(M, N, K))


def gemm_f32_variant_name(variant: int) -> str | None:
    name = load_library().gemm_f32_variant_name(int(variant))
    return name.decode() if name is not None else None


def gemm_f32_status_string(status: int) -> str:
    return load_library().gemm_f32_status_string(int(status)).decode()


def _ld(t: torch.Tensor) -> int:
    if t.dim() != 2 or t.dtype != torch.float32:
        raise TypeError("matrices must be 2-D float32 tensors")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("matrices must be row-major (unit column stride)")
    return max(t.stride(0) if t.shape[0] > 1 else t.shape[1], t.shape[1], 1)


def gemm(A: torch.Tensor, B: torch.Tensor, out: torch.Tensor | None = None,
         variant=None, stream=None, op_a="N", op_b="N") -> torch.Tensor:
    """Tensor form: returns ``out`` (allocated if None) = op(A) @ op(B).  A
    and B are the stored row-major tensors (with op 'T', A is K x M and B is
    N x K); views with a leading dimension (``stride(0)``) and a storage
    offset are passed through as they are.  ``variant`` selects a ladder
    rung and requires op 'N' for both factors."""
    M, K = A.shape if op_a in ("N", 0) else A.shape[::-1]
    K2, N = B.shape if op_b in ("N", 0) else B.shape[::-1]
    if K != K2:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=A.device)
    if tuple(out.shape) != (M, N):
        raise ValueError("out has the wrong shape")
    args = (M, N, K, A, _ld(A), B, _ld(B), out, _ld(out))
    if op_a not in ("N", 0) or op_b not in ("N", 0):
        if variant is not None:
            raise ValueError("transposed factors run on the default kernel only")
        gemm_f32_op(op_a, op_b, *args, stream=stream)
    elif variant is None:
        gemm_f32(*args, stream=stream)
    else:
        gemm_f32_variant(variant, *args, stream=stream)
    return out


def transpose_f32(rows, cols, src, ld_in, dst, ld_out, stream=None) -> None:
    """dst (cols x rows) = src (rows x cols) transposed; see gemm_f32.h."""
    lib = load_library()
    _check(lib.transpose_f32(rows, cols, _addr(src), ld_in, _addr(dst), ld_out, _stream(stream)))


def transpose_f32_variant(variant, rows, cols, src, ld_in, dst, ld_out, stream=None) -> None:
    lib = load_library()
    _check(lib.transpose_f32_variant(int(variant), rows, cols, _addr(src), ld_in, _addr(dst), ld_out,
                                     _stream(stream)))


def transpose_f32_num_variants() -> int:
    return load_library().transpose_f32_num_variants()


def transpose_f32_default_variant(rows, cols, ld_in, ld_out) -> int:
    """The variant transpose_f32 runs for these sizes (-1 for invalid ones)."""
    return int(load_library().transpose_f32_default_variant(rows, cols, ld_in, ld_out))


def transpose_f32_variant_name(variant: int) -> str | None:
    name = load_library().transpose_f32_variant_name(int(variant))
    return name.decode() if name is not None else None


def transpose(X: torch.Tensor, out: torch.Tensor | None = None, variant=None, stream=None) -> torch.Tensor:
    """Tensor form: returns ``out`` (allocated if None) = X^T for a 2-D
    float32 row-major CUDA tensor (views with a leading dimension allowed)."""
    rows, cols = X.shape
    if out is None:
        out = torch.empty((cols, rows), dtype=torch.float32, device=X.device)
    if tuple(out.shape) != (cols, rows):
        raise ValueError("out has the wrong shape")
    args = (rows, cols, X, _ld(X), out, _ld(out))
    if variant is None:
        transpose_f32(*args, stream=stream)
    else:
        transpose_f32_variant(variant, *args, stream=stream)
    return out


def gemm_f32_valu_probe(form, blocks, iters, out, stamps, stream=None) -> None:
    """The vector-ALU FMA loop of the library's measurement helper."""
    lib = load_library()
    _check(lib.gemm_f32_valu_probe(int(form), int(blocks), int(iters), _addr(out), _addr(stamps), _stream(stream)))


def gemm_f32_lds_probe(form, offsets, iters, out, stream=None) -> None:
    """The LDS read probe of the library's measurement helper (offsets: 64
    int32 on the device; out: 64 uint32 or int32 on the device)."""
    lib = load_library()
    _check(lib.gemm_f32_lds_probe(int(form), _addr(offsets), int(iters), _addr(out), _stream(stream)))


def gemm_f32_copy_probe(mode, blocks, iters, src, out, cycles, stream=None) -> None:
    """The copy-rate probe of the library's measurement helper."""
    lib = load_library()
    _check(lib.gemm_f32_copy_probe(int(mode), int(blocks), int(iters), _addr(src), _addr(out), _addr(cycles),
                                   _stream(stream)))


def gemm_f32_ksplit_timeline(M, N, K, A, lda, B, ldb, C, ldc, timeline, timeline_words, stream=None) -> None:
    """gemm_f32's k-split kernel with its per-wave timeline (measurement helper)."""
    lib = load_library()
    _check(lib.gemm_f32_ksplit_timeline(M, N, K, _addr(A), lda, _addr(B), ldb, _addr(C), ldc, _addr(timeline),
                                        int(timeline_words), _stream(stream)))


REDUCE_DEFAULT = 4


def reduce_sum_f32_workspace_size(variant: int, n: int) -> int:
    return load_library().reduce_sum_f32_workspace_size(int(variant), int(n))


def reduce_sum_f32(n, x, out, workspace, workspace_bytes, stream=None) -> None:
    """*out = sum of x[0 .. n-1] (device pointers); see gemm_f32.h."""
    lib = load_library()
    _check(lib.reduce_sum_f32(n, _addr(x), _addr(out), _addr(workspace), workspace_bytes, _stream(stream)))


def reduce_sum_f32_variant(variant, n, x, out, workspace, workspace_bytes, stream=None) -> None:
    lib = load_library()
    _check(lib.reduce_sum_f32_variant(int(variant), n, _addr(x), _addr(out), _addr(workspace),
                                      workspace_bytes, _stream(stream)))


def reduce_sum_f32_variant_noalloc(variant, n, x, out, stream=None) -> None:
    """reduce_sum_f32_variant with the partials in the library's fixed
    per-device scratch (no workspace, no allocation)."""
    lib = load_library()
    _check(lib.reduce_sum_f32_variant_noalloc(int(variant), n, _addr(x), _addr(out), _stream(stream)))


REDUCE_SCRATCH_BYTES = 1 << 20     # REDUCE_SUM_F32_SCRATCH_BYTES


def reduce_sum_f32_num_variants() -> int:
    return load_library().reduce_sum_f32_num_variants()


def reduce_sum_f32_variant_name(variant: int) -> str | None:
    name = load_library().reduce_sum_f32_variant_name(int(variant))
    return name.decode() if name is not None else None


def reduce_sum(x: torch.Tensor, variant=None, stream=None) -> torch.Tensor:
    """Tensor form: a one-element float32 CUDA tensor holding the sum of the
    contiguous float32 tensor x; the workspace is allocated with torch."""
    if x.dtype != torch.float32 or not x.is_contiguous():
        raise TypeError("x must be a contiguous float32 tensor")
    n = x.numel()
    v = REDUCE_DEFAULT if variant is None else int(variant)
    out = torch.empty(1, dtype=torch.float32, device=x.device)
    ws_bytes = reduce_sum_f32_workspace_size(v, n)
    ws = torch.empty(max(ws_bytes // 4, 1), dtype=torch.float32, device=x.device)
    if variant is None:
        reduce_sum_f32(n, x, out, ws, ws_bytes, stream=stream)
    else:
        reduce_sum_f32_variant(v, n, x, out, ws, ws_bytes, stream=stream)
    return out


FORMATS = {"bf16": 0, "f16": 1}
_FORMAT_OF_DTYPE = {torch.bfloat16: 0, torch.float16: 1}


def _format(fmt) -> int:
    if isinstance(fmt, str):
        return FORMATS[fmt]
    return int(fmt)


def gemm_mixed(fmt, M, N, K, A, lda, B, ldb, C, ldc, stream=None) -> None:
    """C (binary32) = A x B for 16-bit A and B of format ``fmt`` ('bf16' or
    'f16'); leading dimensions in elements; see gemm_f32.h."""
    lib = load_library()
    _check(lib.gemm_mixed(_format(fmt), M, N, K, _addr(A), lda, _addr(B), ldb, _addr(C), ldc,
                          _stream(stream)))


def gemm_mixed_variant(variant, fmt, M, N, K, A, lda, B, ldb, C, ldc, stream=None) -> None:
    lib = load_library()
    _check(lib.gemm_mixed_variant(int(variant), _format(fmt), M, N, K, _addr(A), lda, _addr(B), ldb,
                                  _addr(C), ldc, _stream(stream)))


def gemm_mixed_op(op_a, op_b, fmt, M, N, K, A, lda, B, ldb, C, ldc, stream=None) -> None:
    """C (binary32) = op(A) x op(B) for 16-bit factors, op 'N' (as stored) or
    'T' (stored transposed: A is K x M, B is N x K); see gemm_f32.h."""
    lib = load_library()
    oa = OPS.get(op_a, op_a) if not isinstance(op_a, int) else op_a
    ob = OPS.get(op_b, op_b) if not isinstance(op_b, int) else op_b
    _check(lib.gemm_mixed_op(int(oa), int(ob), _format(fmt), M, N, K, _addr(A), lda, _addr(B), ldb,
                             _addr(C), ldc, _stream(stream)))


def gemm_mixed_num_variants() -> int:
    return load_library().gemm_mixed_num_variants()


def gemm_mixed_default_variant(M, N, K) -> int:
    """The configuration gemm_mixed runs for M x N x K (-1 for invalid
    sizes); no device needed."""
    return int(load_library().gemm_mixed_default_variant(M, N, K))


def gemm_mixed_variant_name(variant: int) -> str | None:
    name = load_library().gemm_mixed_variant_name(int(variant))
    return name.decode() if name is not None else None


def _ld16(t: torch.Tensor) -> int:
    if t.dim() != 2 or t.dtype not in _FORMAT_OF_DTYPE:
        raise TypeError("16-bit factors must be 2-D bfloat16 or float16 tensors")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("matrices must be row-major (unit column stride)")
    return max(t.stride(0) if t.shape[0] > 1 else t.shape[1], t.shape[1], 1)


def gemm16(A: torch.Tensor, B: torch.Tensor, out: torch.Tensor | None = None, variant=None,
           stream=None, op_a="N", op_b="N") -> torch.Tensor:
    """Tensor form: returns ``out`` (float32, allocated if None) = op(A) @
    op(B) for bfloat16 or float16 CUDA tensors of one dtype.  A and B are the
    stored row-major tensors (with op 'T', A is K x M and B is N x K); views
    with a leading dimension and a storage offset pass through.  ``variant``
    selects a tile configuration and requires op 'N' for both factors."""
    if A.dtype != B.dtype:
        raise TypeError("A and B must have the same 16-bit dtype")
    M, K = A.shape if op_a in ("N", 0) else A.shape[::-1]
    K2, N = B.shape if op_b in ("N", 0) else B.shape[::-1]
    if K != K2:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=A.device)
    if tuple(out.shape) != (M, N):
        raise ValueError("out has the wrong shape")
    args = (_FORMAT_OF_DTYPE[A.dtype], M, N, K, A, _ld16(A), B, _ld16(B), out, _ld(out))
    if op_a not in ("N", 0) or op_b not in ("N", 0):
        if variant is not None:
            raise ValueError("transposed factors run on the default kernels only")
        gemm_mixed_op(op_a, op_b, *args, stream=stream)
    elif variant is None:
        gemm_mixed(*args, stream=stream)
    else:
        gemm_mixed_variant(variant, *args, stream=stream)
    return out


# ------------------------------------------------- layers: product + epilogue

TYPES = {"bf16": 0, "f16": 1, "f32": 2}
_TYPE_OF_DTYPE = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}


def _activation(activation) -> int:
    if activation is None:
        return 0
    if isinstance(activation, str):
        if activation not in ACTIVATIONS:
            raise ValueError(f"unknown activation {activation!r}")
        return ACTIVATIONS[activation]
    return int(activation)


def epilogue(c_type, activation=0, gradient=0, bias=None, bias_type=0, residual=None, ld_residual=0, preact=None,
             ld_preact=0, bias_grad=None) -> Epilogue:
    """A gemm_epilogue; pointers as tensors or device addresses."""
    return Epilogue(int(c_type), _activation(activation), int(gradient), int(bias_type), _addr(bias), _addr(residual),
                    int(ld_residual), _addr(preact), int(ld_preact), _addr(bias_grad))


def gemm_mixed_epilogue_workspace_size(op_a, op_b, fmt, M, N, K, A, lda, B, ldb, ep: Epilogue) -> int:
    return int(load_library().gemm_mixed_epilogue_workspace_size(
        int(OPS.get(op_a, op_a)), int(OPS.get(op_b, op_b)), _format(fmt), M, N, K, _addr(A), lda, _addr(B), ldb,
        ctypes.byref(ep)))


def gemm_mixed_epilogue(op_a, op_b, fmt, M, N, K, A, lda, B, ldb, C, ldc, ep: Epilogue, workspace=None,
                        workspace_bytes=0, stream=None) -> None:
    """The 16-bit product with its epilogue; see gemm_f32.h."""
    _check(load_library().gemm_mixed_epilogue(
        int(OPS.get(op_a, op_a)), int(OPS.get(op_b, op_b)), _format(fmt), M, N, K, _addr(A), lda, _addr(B), ldb,
        _addr(C), ldc, ctypes.byref(ep), _addr(workspace), workspace_bytes, _stream(stream)))


def activation_grad_workspace_size(M, N) -> int:
    return int(load_library().activation_grad_workspace_size(M, N))


def activation_grad(activation, fmt, M, N, dY, ld_dy, preact, ld_preact, dZ, ld_dz, bias_grad, workspace=None,
                    workspace_bytes=0, stream=None) -> None:
    """dZ = dY * act'(Z) and its column sums; see gemm_f32.h."""
    _check(load_library().activation_grad(_activation(activation), _format(fmt), M, N, _addr(dY), ld_dy,
                                          _addr(preact), ld_preact, _addr(dZ), ld_dz, _addr(bias_grad),
                                          _addr(workspace), workspace_bytes, _stream(stream)))


def layer_norm_backward_workspace_size(type_, rows, cols) -> int:
    return int(load_library().layer_norm_backward_workspace_size(int(type_), rows, cols))


def newton_schulz_workspace_size(type_, batch, rows, cols) -> int:
    return int(load_library().newton_schulz_workspace_size(int(type_), batch, rows, cols))


def _device_of(*tensors) -> int:
    """Index of the one GPU that holds all the tensors (None ones aside)."""
    device = None
    for t in tensors:
        if t is None:
            continue
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError("arguments must be CUDA tensors")
        if device is None:
            device = t.get_device()
        elif t.get_device() != device:
            raise ValueError(f"tensors on different devices: cuda:{device} and {t.device}")
    return device


def _elsewhere(stream, device: int) -> bool:
    """Whether a call has to change torch's current stream or device first."""
    return stream is not None or device != torch._C._cuda_getDevice()


@contextlib.contextmanager
def _placed(stream, device: int):
    """The tensors' device current and, if a stream is given, that stream
    torch's current one: outputs and workspaces allocated inside belong to the
    stream the kernels run on."""
    if stream is None:
        with torch.cuda.device(device):
            yield
        return
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    if stream.device.index != device:
        raise ValueError(f"stream of {stream.device} for tensors on cuda:{device}")
    with torch.cuda.stream(stream):
        yield


def _workspace(like: torch.Tensor, nbytes: int):
    """(tensor, address, bytes) of a workspace of torch's; a size of -1 is
    left for the call itself to name the error."""
    if nbytes <= 0:
        return None, None, 0
    ws = like.new_empty(nbytes, dtype=torch.uint8)
    return ws, ws.data_ptr(), nbytes


def _row_major(t: torch.Tensor, what: str) -> int:
    """Leading dimension of a row-major matrix, or of each of a batch of them."""
    rows, cols = t.shape[-2:]
    s0, s1 = t.stride()[-2:]
    if cols > 1 and s1 != 1:
        raise ValueError(f"{what} must be row-major (unit column stride)")
    if rows <= 1:
        return cols or 1
    if s0 < cols:
        raise ValueError(f"{what}'s rows overlap (row stride {s0}, {cols} columns)")
    return s0 or 1


def _matrix(t: torch.Tensor, what: str, rows: int, cols: int, dtype) -> int:
    """Leading dimension of a matrix argument of known shape and dtype."""
    if t.dim() != 2 or t.dtype is not dtype:
        raise TypeError(f"{what} must be a 2-D tensor of {dtype}")
    if t.shape[0] != rows or t.shape[1] != cols:
        raise ValueError(f"{what} has shape {tuple(t.shape)}, not {(rows, cols)}")
    return _row_major(t, what)


def _vector(t: torch.Tensor, what: str, n: int, dtypes) -> None:
    if t.dim() != 1 or t.shape[0] != n or not t.is_contiguous() or t.dtype not in dtypes:
        raise TypeError(f"{what} must be a contiguous vector of {n} values of {', '.join(str(d) for d in dtypes)}")


def _factors(A, B, op_a, op_b):
    """(format, op_a, op_b, M, N, K, lda, ldb) of a 16-bit product's factors."""
    oa, ob = OPS[op_a], OPS[op_b]
    fmt = _FORMAT_OF_DTYPE.get(A.dtype)
    if fmt is None or B.dtype is not A.dtype or A.dim() != 2 or B.dim() != 2:
        raise TypeError("the factors must be 2-D bfloat16 or float16 tensors of one dtype")
    lda, ldb = _row_major(A, "the first factor"), _row_major(B, "the second factor")
    M, K = A.shape
    K2, N = B.shape
    if oa:
        M, K = K, M
    if ob:
        K2, N = N, K2
    if K != K2:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    return fmt, oa, ob, M, N, K, lda, ldb


def _output(out, out_dtype, like: torch.Tensor, M: int, N: int):
    """(out, its leading dimension), allocated if None."""
    if out is None:
        dtype = out_dtype or like.dtype
        if dtype is not like.dtype and dtype is not torch.float32:
            raise TypeError(f"out has the factors' dtype or float32, not {dtype}")
        return (like.new_empty((M, N)) if dtype is like.dtype else like.new_empty((M, N), dtype=dtype)), N or 1
    if out_dtype is not None and out.dtype is not out_dtype:
        raise TypeError(f"out is {out.dtype}, not {out_dtype}")
    return out, _matrix(out, "out", M, N, torch.float32 if out.dtype is torch.float32 else like.dtype)


def _linear_call(fmt, oa, ob, M, N, K, A, lda, B, ldb, C, ldc, ep) -> None:
    """gemm_mixed_epilogue on the current stream with a workspace of torch's."""
    lib = load_library()
    a, b, ref = A.data_ptr(), B.data_ptr(), ctypes.byref(ep)
    ws, addr, nbytes = _workspace(A, lib.gemm_mixed_epilogue_workspace_size(oa, ob, fmt, M, N, K, a, lda, b, ldb, ref))
    _check(lib.gemm_mixed_epilogue(oa, ob, fmt, M, N, K, a, lda, b, ldb, C.data_ptr(), ldc, ref, addr, nbytes,
                                   torch._C._cuda_getCurrentRawStream(A.get_device())))


def linear(X, W, bias=None, activation="none", residual=None, out=None, out_dtype=None, return_preact=False,
           op_a="N", op_b="N", stream=None):
    """act(op_a(X) @ op_b(W) + bias) + residual for bfloat16 or float16 X and
    W, with the rest in the product kernel's epilogue (few rows or tiles with a
    long K: in a pass over binary32 partial sums).

    ``op_b="T"``: W is stored N x K.  ``out`` (or ``out_dtype``) has the
    factors' dtype (default) or float32 and overlaps neither of them;
    ``residual`` has out's dtype and may be ``out``; ``bias`` has the factors' dtype or float32.  With
    ``return_preact`` returns (out, Z), Z = op_a(X) @ op_b(W) + bias in the
    factors' dtype, for the backward pass."""
    device = _device_of(X, W, bias, residual, out)
    if _elsewhere(stream, device):
        with _placed(stream, device):
            return linear(X, W, bias, activation, residual, out, out_dtype, return_preact, op_a, op_b)
    fmt, oa, ob, M, N, K, lda, ldb = _factors(X, W, op_a, op_b)
    out, ldc = _output(out, out_dtype, X, M, N)
    c_type = _TYPE_OF_DTYPE[out.dtype]
    ep = Epilogue(c_type, _activation(activation))
    if bias is not None:
        _vector(bias, "bias", N, (X.dtype, torch.float32))
        ep.bias_type = _TYPE_OF_DTYPE[bias.dtype]
        ep.bias = bias.data_ptr()
    if residual is not None:
        ep.ld_residual = _matrix(residual, "residual", M, N, out.dtype)
        ep.residual = residual.data_ptr()
    preact = None
    if return_preact:
        preact = X.new_empty((M, N))
        ep.preact = preact.data_ptr()
        ep.ld_preact = N or 1
    _linear_call(fmt, oa, ob, M, N, K, X, lda, W, ldb, out, ldc, ep)
    return (out, preact) if return_preact else out


def linear_grad(dZ, W, preact=None, activation="none", residual=None, out=None, out_dtype=None,
                return_bias_grad=False, op_a="N", op_b="T", stream=None):
    """(op_a(dZ) @ op_b(W) + residual) * act'(preact): the gradient that a
    layer passes to the one before it, through that layer's activation.

    With the defaults dZ is M x N and W the K x N weight of
    ``linear(X, W)``, the result M x K; ``preact`` is what
    ``linear(..., return_preact=True)`` of the layer before returned,
    ``residual`` a gradient that arrives past this layer (out's dtype; may be
    ``out``, which overlaps no other argument).  With
    ``return_bias_grad`` returns (out, column sums in float32): the bias
    gradient of the layer before."""
    device = _device_of(dZ, W, preact, residual, out)
    if _elsewhere(stream, device):
        with _placed(stream, device):
            return linear_grad(dZ, W, preact, activation, residual, out, out_dtype, return_bias_grad, op_a, op_b)
    fmt, oa, ob, M, N, K, lda, ldb = _factors(dZ, W, op_a, op_b)
    out, ldc = _output(out, out_dtype, dZ, M, N)
    act = _activation(activation)
    if preact is None and act:
        raise ValueError("the gradient of an activation needs preact")
    ep = Epilogue(_TYPE_OF_DTYPE[out.dtype], act, 1)
    if preact is not None:
        ep.ld_preact = _matrix(preact, "preact", M, N, dZ.dtype)
        ep.preact = preact.data_ptr()
    if residual is not None:
        ep.ld_residual = _matrix(residual, "residual", M, N, out.dtype)
        ep.residual = residual.data_ptr()
    sums = None
    if return_bias_grad:
        sums = dZ.new_empty(N, dtype=torch.float32)
        ep.bias_grad = sums.data_ptr()
    _linear_call(fmt, oa, ob, M, N, K, dZ, lda, W, ldb, out, ldc, ep)
    return (out, sums) if return_bias_grad else out


def activation_backward(dY, preact=None, activation="none", out=None, return_bias_grad=True, return_dz=True,
                        stream=None):
    """(dZ, db): dZ = dY * act'(preact) in dY's dtype, db its column sums in
    float32 (None without ``return_bias_grad``); with ``return_dz`` false only
    the sums are computed and dZ is None.  ``out`` may be dY."""
    device = _device_of(dY, preact, out)
    if _elsewhere(stream, device):
        with _placed(stream, device):
            return activation_backward(dY, preact, activation, out, return_bias_grad, return_dz)
    lib = load_library()
    fmt = _FORMAT_OF_DTYPE.get(dY.dtype)
    if fmt is None or dY.dim() != 2:
        raise TypeError("dY must be a 2-D bfloat16 or float16 tensor")
    ldy = _row_major(dY, "dY")
    M, N = dY.shape
    act = _activation(activation)
    if preact is None and act:
        raise ValueError("the gradient of an activation needs preact")
    ldz = 0 if preact is None else _matrix(preact, "preact", M, N, dY.dtype)
    if not return_dz:
        out, ldo = None, 0
    elif out is None:
        out, ldo = dY.new_empty((M, N)), N or 1
    else:
        ldo = _matrix(out, "out", M, N, dY.dtype)
    sums, ws, addr, nbytes = None, None, None, 0
    if return_bias_grad:
        sums = dY.new_empty(N, dtype=torch.float32)
        ws, addr, nbytes = _workspace(dY, lib.activation_grad_workspace_size(M, N))
    _check(lib.activation_grad(act, fmt, M, N, dY.data_ptr(), ldy, _addr(preact), ldz, _addr(out), ldo, _addr(sums),
                               addr, nbytes, torch._C._cuda_getCurrentRawStream(device)))
    return out, sums


def linear_backward(dY, X, W, preact=None, activation="none", weight_grad_dtype=None, op_b="N", stream=None,
                    return_bias_grad=True):
    """(dX, dW, db) of Y = act(X @ op_b(W) + bias): dZ = dY * act'(preact), db
    its column sums (float32), dX = dZ @ op_b(W)^T in dY's dtype, dW in W's
    layout and dtype (or float32 with ``weight_grad_dtype``).  dZ is rounded
    to dY's dtype between the two, for the matrix units.  The gradient of a
    residual added after the activation is dY itself.  Without
    ``return_bias_grad`` (a layer that has no bias) db is None, and without an
    activation dY is then read by the products only."""
    device = _device_of(dY, X, W, preact)
    if _elsewhere(stream, device):
        with _placed(stream, device):
            return linear_backward(dY, X, W, preact, activation, weight_grad_dtype, op_b, None, return_bias_grad)
    fmt, _, ob, M, N, K, ldx, ldw = _factors(X, W, "N", op_b)
    lddz = _matrix(dY, "dY", M, N, X.dtype)
    if weight_grad_dtype not in (None, W.dtype, torch.float32):
        raise TypeError("dW has W's dtype or float32")
    if _activation(activation):
        dZ, db = activation_backward(dY, preact, activation, return_bias_grad=return_bias_grad)
        lddz = N or 1
    else:
        dZ = dY
        db = activation_backward(dY, return_dz=False)[1] if return_bias_grad else None
    dX = dY.new_empty((M, K))
    _linear_call(fmt, 0, 1 - ob, M, K, N, dZ, lddz, W, ldw, dX, K or 1, Epilogue(fmt))
    dW, lddw = _output(None, weight_grad_dtype, W, *W.shape)
    ep = Epilogue(_TYPE_OF_DTYPE[dW.dtype])
    if ob:
        _linear_call(fmt, 1, 0, N, K, M, dZ, lddz, X, ldx, dW, lddw, ep)
    else:
        _linear_call(fmt, 1, 0, K, N, M, X, ldx, dZ, lddz, dW, lddw, ep)
    return dX, dW, db


# ------------------------------------------------------------- layer norm

def layer_norm(X, weight=None, bias=None, eps=1e-5, out=None, stream=None):
    """(Y, mean, rstd) of the layer norm over X's rows (2-D, bfloat16, float16
    or float32; Y of X's dtype, mean and rstd float32).  ``weight`` and
    ``bias`` are vectors of one dtype of the three; ``out`` may be X."""
    device = _device_of(X, weight, bias, out)
    if _elsewhere(stream, device):
        with _placed(stream, device):
            return layer_norm(X, weight, bias, eps, out)
    t = _TYPE_OF_DTYPE.get(X.dtype)
    if t is None or X.dim() != 2:
        raise TypeError("X must be a 2-D bfloat16, float16 or float32 tensor")
    ldx = _row_major(X, "X")
    rows, cols = X.shape
    param, gamma, beta = 2, None, None
    if weight is not None:
        _vector(weight, "weight", cols, _TYPE_OF_DTYPE)
        param, gamma = _TYPE_OF_DTYPE[weight.dtype], weight.data_ptr()
    if bias is not None:
        _vector(bias, "bias", cols, _TYPE_OF_DTYPE if weight is None else (weight.dtype,))
        param, beta = _TYPE_OF_DTYPE[bias.dtype], bias.data_ptr()
    if out is None:
        out, ldy = X.new_empty((rows, cols)), cols
    else:
        ldy = _matrix(out, "out", rows, cols, X.dtype)
    mean, rstd = X.new_empty(rows, dtype=torch.float32), X.new_empty(rows, dtype=torch.float32)
    _check(load_library().layer_norm(t, rows, cols, X.data_ptr(), ldx, param, gamma, beta, eps, out.data_ptr(), ldy,
                                     mean.data_ptr(), rstd.data_ptr(), torch._C._cuda_getCurrentRawStream(device)))
    return out, mean, rstd


def layer_norm_backward(dY, X, mean, rstd, weight=None, residual_grad=None, out=None, stream=None,
                        return_param_grads=True):
    """(dX, dweight, dbias) of layer_norm; ``residual_grad`` (dY's dtype) is
    added to dX.  dweight and dbias are float32, None without
    ``return_param_grads`` (a norm that has no parameters).  ``out`` may be dY
    or ``residual_grad``."""
    device = _device_of(dY, X, mean, rstd, weight, residual_grad, out)
    if _elsewhere(stream, device):
        with _placed(stream, device):
            return layer_norm_backward(dY, X, mean, rstd, weight, residual_grad, out, None, return_param_grads)
    lib = load_library()
    t = _TYPE_OF_DTYPE.get(dY.dtype)
    if t is None or dY.dim() != 2:
        raise TypeError("dY must be a 2-D bfloat16, float16 or float32 tensor")
    lddy = _row_major(dY, "dY")
    rows, cols = dY.shape
    ldx = _matrix(X, "X", rows, cols, dY.dtype)
    _vector(mean, "mean", rows, (torch.float32,))
    _vector(rstd, "rstd", rows, (torch.float32,))
    param, gamma, rgrad, ldr = 2, None, None, 0
    if weight is not None:
        _vector(weight, "weight", cols, _TYPE_OF_DTYPE)
        param, gamma = _TYPE_OF_DTYPE[weight.dtype], weight.data_ptr()
    if residual_grad is not None:
        ldr = _matrix(residual_grad, "residual_grad", rows, cols, dY.dtype)
        rgrad = residual_grad.data_ptr()
    if out is None:
        out, lddx = dY.new_empty((rows, cols)), cols
    else:
        lddx = _matrix(out, "out", rows, cols, dY.dtype)
    dweight, dbias, ws, addr, nbytes = None, None, None, None, 0
    if return_param_grads:
        dweight, dbias = dY.new_empty(cols, dtype=torch.float32), dY.new_empty(cols, dtype=torch.float32)
        ws, addr, nbytes = _workspace(dY, lib.layer_norm_backward_workspace_size(t, rows, cols))
    _check(lib.layer_norm_backward(t, rows, cols, dY.data_ptr(), lddy, X.data_ptr(), ldx, mean.data_ptr(),
                                   rstd.data_ptr(), param, gamma, rgrad, ldr, out.data_ptr(), lddx,
                                   _addr(dweight), _addr(dbias), addr, nbytes,
                                   torch._C._cuda_getCurrentRawStream(device)))
    return out, dweight, dbias


# ---------------------------------------------------------- Newton-Schulz

NEWTON_SCHULZ_COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def newton_schulz(G, steps=5, coefficients=NEWTON_SCHULZ_COEFFICIENTS, eps=1e-7, out=None, stream=None):
    """The matrix G (2-D, or 3-D: a batch of matrices of one shape; bfloat16,
    float16 or float32) orthogonalised by ``steps`` Newton-Schulz steps of the
    odd polynomial with ``coefficients`` (a, b, c); see gemm_f32.h.  Accurate
    relative to the matrix: entries below 2^-39 of its norm count as 0.
    ``out`` (G's shape and dtype) may be G."""
    device = _device_of(G, out)
    if _elsewhere(stream, device):
        with _placed(stream, device):
            return newton_schulz(G, steps, coefficients, eps, out)
    lib = load_library()
    t = _TYPE_OF_DTYPE.get(G.dtype)
    if t is None or G.dim() not in (2, 3):
        raise TypeError("G must be a 2-D or 3-D bfloat16, float16 or float32 tensor")
    if out is None:
        out = G.new_empty(G.shape)
    elif out.shape != G.shape or out.dtype is not G.dtype:
        raise ValueError("out must have G's shape and dtype")
    batch = G.shape[0] if G.dim() == 3 else 1
    rows, cols = G.shape[-2:]

    def strides(m, what):
        ld = _row_major(m, what)
        return ld, (m.stride(0) if m.dim() == 3 and batch > 1 else max(rows - 1, 0) * ld + cols)

    ldg, stride_g = strides(G, "G")
    ldo, stride_o = strides(out, "out")
    a, b, c = (float(v) for v in coefficients)
    ws, addr, nbytes = _workspace(G, lib.newton_schulz_workspace_size(t, batch, rows, cols))
    _check(lib.newton_schulz(t, batch, rows, cols, G.data_ptr(), ldg, stride_g, int(steps), a, b, c, float(eps),
                             out.data_ptr(), ldo, stride_o, addr, nbytes, torch._C._cuda_getCurrentRawStream(device)))
    return out
