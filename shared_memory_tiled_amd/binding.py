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


class _Launch:
    """Makes the tensors' device current and, if a stream is given, that
    stream torch's current one, so that outputs and workspaces allocated
    inside belong to the stream the kernels run on; ``handle`` is that
    stream.  All tensors must live on one GPU."""

    def __init__(self, stream, *tensors):
        device = None
        for t in tensors:
            if t is None:
                continue
            if not isinstance(t, torch.Tensor) or not t.is_cuda:
                raise TypeError("arguments must be CUDA tensors")
            if device is None:
                device = t.device
            elif t.device != device:
                raise ValueError(f"tensors on different devices: {device} and {t.device}")
        self.device = device
        if stream is not None and not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), device=device)
        if stream is not None and stream.device != device:
            raise ValueError(f"stream of {stream.device} for tensors on {device}")
        self._stream = stream
        self._contexts = []

    def __enter__(self):
        if self._stream is not None:
            self._contexts = [torch.cuda.stream(self._stream)]
        elif torch.cuda.current_device() != self.device.index:
            self._contexts = [torch.cuda.device(self.device)]
        for c in self._contexts:
            c.__enter__()
        self.handle = torch.cuda.current_stream(self.device).cuda_stream
        return self

    def __exit__(self, *exc):
        for c in reversed(self._contexts):
            c.__exit__(*exc)
        return False

    def workspace(self, nbytes: int):
        if nbytes < 0:
            raise GemmError(6, "the library takes no problem of this size")
        return torch.empty(nbytes, dtype=torch.uint8, device=self.device) if nbytes else None


def _ld_any(t: torch.Tensor, what: str, shape=None, dtypes=None) -> int:
    """Leading dimension of a row-major matrix argument, after its checks."""
    if t.dim() != 2 or (dtypes is not None and t.dtype not in dtypes):
        raise TypeError(f"{what} must be a 2-D tensor of {', '.join(str(d) for d in dtypes or ())}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} has shape {tuple(t.shape)}, not {tuple(shape)}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{what} must be row-major (unit column stride)")
    ld = t.stride(0) if t.shape[0] > 1 else t.shape[1]
    if t.shape[0] > 1 and ld < t.shape[1]:
        raise ValueError(f"{what}'s rows overlap (row stride {ld}, {t.shape[1]} columns)")
    return max(ld, t.shape[1], 1)


def _vector(t: torch.Tensor | None, what: str, n: int, dtypes) -> None:
    if t is None:
        return
    if t.dim() != 1 or t.shape[0] != n or not t.is_contiguous() or t.dtype not in dtypes:
        raise TypeError(f"{what} must be a contiguous vector of {n} values of {', '.join(str(d) for d in dtypes)}")


def _linear_call(launch, op_a, op_b, M, N, K, A, lda, B, ldb, C, ldc, ep) -> None:
    """gemm_mixed_epilogue with a workspace of torch's."""
    lib = load_library()
    fmt = _FORMAT_OF_DTYPE[A.dtype]
    head = (op_a, op_b, fmt, M, N, K, A.data_ptr(), lda, B.data_ptr(), ldb)
    ref = ctypes.byref(ep)
    nbytes = lib.gemm_mixed_epilogue_workspace_size(*head, ref)
    ws = launch.workspace(nbytes) if nbytes > 0 else None          # -1: the call itself names the error
    _check(lib.gemm_mixed_epilogue(*head, C.data_ptr(), ldc, ref, None if ws is None else ws.data_ptr(),
                                   max(nbytes, 0), launch.handle))


def _factors(A, B, op_a, op_b):
    """(op_a, op_b, M, N, K, lda, ldb) of a 16-bit product's checked factors."""
    oa, ob = int(OPS[op_a]), int(OPS[op_b])
    dt = tuple(_FORMAT_OF_DTYPE)
    lda, ldb = _ld_any(A, "the first factor", dtypes=dt), _ld_any(B, "the second factor", dtypes=dt)
    if A.dtype != B.dtype:
        raise TypeError("the factors must have the same 16-bit dtype")
    M, K = A.shape[::-1] if oa else A.shape
    K2, N = B.shape[::-1] if ob else B.shape
    if K != K2:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    return oa, ob, M, N, K, lda, ldb


def linear(X, W, bias=None, activation="none", residual=None, out=None, out_dtype=None, return_preact=False,
           op_a="N", op_b="N", stream=None):
    """act(op_a(X) @ op_b(W) + bias) + residual for bfloat16 or float16 X and
    W, in one product kernel with the rest in its epilogue.

    ``op_b="T"``: W is stored N x K.  ``out`` (or ``out_dtype``) has the
    factors' dtype (default) or float32; ``residual`` has out's dtype and may
    be ``out``; ``bias`` has the factors' dtype or float32.  With
    ``return_preact`` returns (out, Z), Z = op_a(X) @ op_b(W) + bias in the
    factors' dtype, for the backward pass."""
    with _Launch(stream, X, W, bias, residual, out) as launch:
        oa, ob, M, N, K, lda, ldb = _factors(X, W, op_a, op_b)
        if out is None:
            out = torch.empty((M, N), dtype=out_dtype or X.dtype, device=X.device)
        elif out_dtype is not None and out.dtype != out_dtype:
            raise TypeError(f"out is {out.dtype}, not {out_dtype}")
        ldc = _ld_any(out, "out", (M, N), (X.dtype, torch.float32))
        _vector(bias, "bias", N, (X.dtype, torch.float32))
        ldr = 0 if residual is None else _ld_any(residual, "residual", (M, N), (out.dtype,))
        preact = torch.empty((M, N), dtype=X.dtype, device=X.device) if return_preact else None
        ep = epilogue(_TYPE_OF_DTYPE[out.dtype], activation, 0, bias,
                      0 if bias is None else _TYPE_OF_DTYPE[bias.dtype], residual, ldr, preact, max(N, 1))
        _linear_call(launch, oa, ob, M, N, K, X, lda, W, ldb, out, ldc, ep)
    return (out, preact) if return_preact else out


def linear_grad(dZ, W, preact=None, activation="none", residual=None, out=None, out_dtype=None,
                return_bias_grad=False, op_a="N", op_b="T", stream=None):
    """(op_a(dZ) @ op_b(W) + residual) * act'(preact): the gradient that a
    layer passes to the one before it, through that layer's activation.

    With the defaults dZ is M x N and W the K x N weight of
    ``linear(X, W)``, the result M x K; ``preact`` is what
    ``linear(..., return_preact=True)`` of the layer before returned,
    ``residual`` a gradient that arrives past this layer (out's dtype).  With
    ``return_bias_grad`` returns (out, column sums in float32): the bias
    gradient of the layer before."""
    with _Launch(stream, dZ, W, preact, residual, out) as launch:
        oa, ob, M, N, K, lda, ldb = _factors(dZ, W, op_a, op_b)
        if out is None:
            out = torch.empty((M, N), dtype=out_dtype or dZ.dtype, device=dZ.device)
        elif out_dtype is not None and out.dtype != out_dtype:
            raise TypeError(f"out is {out.dtype}, not {out_dtype}")
        ldc = _ld_any(out, "out", (M, N), (dZ.dtype, torch.float32))
        if preact is None and _activation(activation):
            raise ValueError("the gradient of an activation needs preact")
        ldz = 0 if preact is None else _ld_any(preact, "preact", (M, N), (dZ.dtype,))
        ldr = 0 if residual is None else _ld_any(residual, "residual", (M, N), (out.dtype,))
        sums = torch.empty(N, dtype=torch.float32, device=dZ.device) if return_bias_grad else None
        ep = epilogue(_TYPE_OF_DTYPE[out.dtype], activation, 1, None, 0, residual, ldr, preact, ldz, sums)
        _linear_call(launch, oa, ob, M, N, K, dZ, lda, W, ldb, out, ldc, ep)
    return (out, sums) if return_bias_grad else out


def activation_backward(dY, preact=None, activation="none", out=None, return_bias_grad=True, return_dz=True,
                        stream=None):
    """(dZ, db): dZ = dY * act'(preact) in dY's dtype, db its column sums in
    float32 (None without ``return_bias_grad``); with ``return_dz`` false only
    the sums are computed and dZ is None.  ``out`` may be dY."""
    with _Launch(stream, dY, preact, out) as launch:
        lib = load_library()
        ldy = _ld_any(dY, "dY", None, tuple(_FORMAT_OF_DTYPE))
        M, N = dY.shape
        act = _activation(activation)
        if preact is None and act:
            raise ValueError("the gradient of an activation needs preact")
        ldz = 0 if preact is None else _ld_any(preact, "preact", (M, N), (dY.dtype,))
        if not return_dz:
            out = None
        elif out is None:
            out = torch.empty((M, N), dtype=dY.dtype, device=dY.device)
        ldo = 0 if out is None else _ld_any(out, "out", (M, N), (dY.dtype,))
        sums = torch.empty(N, dtype=torch.float32, device=dY.device) if return_bias_grad else None
        nbytes = lib.activation_grad_workspace_size(M, N) if return_bias_grad else 0
        ws = launch.workspace(nbytes)
        _check(lib.activation_grad(act, _FORMAT_OF_DTYPE[dY.dtype], M, N, dY.data_ptr(), ldy, _addr(preact), ldz,
                                   _addr(out), ldo, _addr(sums), _addr(ws), nbytes, launch.handle))
    return out, sums


def linear_backward(dY, X, W, preact=None, activation="none", weight_grad_dtype=None, op_b="N", stream=None):
    """(dX, dW, db) of Y = act(X @ op_b(W) + bias): dZ = dY * act'(preact), db
    its column sums (float32), dX = dZ @ op_b(W)^T in dY's dtype, dW in W's
    layout and dtype (or float32 with ``weight_grad_dtype``).  dZ is rounded
    to dY's dtype between the two, for the matrix units.  The gradient of a
    residual added after the activation is dY itself."""
    with _Launch(stream, dY, X, W, preact) as launch:
        ob = int(OPS[op_b])
        M, N = dY.shape
        dt = (dY.dtype,)
        ldx = _ld_any(X, "X", (M, X.shape[-1]), dt)
        K = X.shape[1]
        ldw = _ld_any(W, "W", (N, K) if ob else (K, N), dt)
        if _activation(activation):
            dZ, db = activation_backward(dY, preact, activation)
        else:
            dZ = dY
            _, db = activation_backward(dY, return_dz=False)
        lddz = _ld_any(dZ, "dY", (M, N), tuple(_FORMAT_OF_DTYPE))
        dX = torch.empty((M, K), dtype=dY.dtype, device=dY.device)
        ep = epilogue(_TYPE_OF_DTYPE[dX.dtype])
        _linear_call(launch, 0, 1 - ob, M, K, N, dZ, lddz, W, ldw, dX, max(K, 1), ep)
        dW = torch.empty(tuple(W.shape), dtype=weight_grad_dtype or W.dtype, device=W.device)
        if dW.dtype not in (W.dtype, torch.float32):
            raise TypeError("dW has W's dtype or float32")
        ep = epilogue(_TYPE_OF_DTYPE[dW.dtype])
        if ob:
            _linear_call(launch, 1, 0, N, K, M, dZ, lddz, X, ldx, dW, max(K, 1), ep)
        else:
            _linear_call(launch, 1, 0, K, N, M, X, ldx, dZ, lddz, dW, max(N, 1), ep)
    return dX, dW, db


# ------------------------------------------------------------- layer norm

def layer_norm(X, weight=None, bias=None, eps=1e-5, out=None, stream=None):
    """(Y, mean, rstd) of the layer norm over X's rows (2-D, bfloat16, float16
    or float32; Y of X's dtype, mean and rstd float32).  ``weight`` and
    ``bias`` are vectors of one dtype of the three; ``out`` may be X."""
    with _Launch(stream, X, weight, bias, out) as launch:
        ldx = _ld_any(X, "X", None, tuple(_TYPE_OF_DTYPE))
        rows, cols = X.shape
        _vector(weight, "weight", cols, tuple(_TYPE_OF_DTYPE))
        _vector(bias, "bias", cols, tuple(_TYPE_OF_DTYPE) if weight is None else (weight.dtype,))
        if out is None:
            out = torch.empty((rows, cols), dtype=X.dtype, device=X.device)
        ldy = _ld_any(out, "out", (rows, cols), (X.dtype,))
        stats = torch.empty((2, rows), dtype=torch.float32, device=X.device)
        param = weight if weight is not None else bias
        _check(load_library().layer_norm(
            _TYPE_OF_DTYPE[X.dtype], rows, cols, X.data_ptr(), ldx, 2 if param is None else _TYPE_OF_DTYPE[param.dtype],
            _addr(weight), _addr(bias), float(eps), out.data_ptr(), ldy, stats.data_ptr(),
            stats.data_ptr() + 4 * rows, launch.handle))
    return out, stats[0], stats[1]


def layer_norm_backward(dY, X, mean, rstd, weight=None, residual_grad=None, out=None, stream=None):
    """(dX, dweight, dbias) of layer_norm; ``residual_grad`` (dY's dtype) is
    added to dX.  dweight and dbias are float32.  ``out`` may be dY or
    ``residual_grad``."""
    with _Launch(stream, dY, X, mean, rstd, weight, residual_grad, out) as launch:
        lib = load_library()
        lddy = _ld_any(dY, "dY", None, tuple(_TYPE_OF_DTYPE))
        rows, cols = dY.shape
        ldx = _ld_any(X, "X", (rows, cols), (dY.dtype,))
        _vector(mean, "mean", rows, (torch.float32,))
        _vector(rstd, "rstd", rows, (torch.float32,))
        _vector(weight, "weight", cols, tuple(_TYPE_OF_DTYPE))
        ldr = 0 if residual_grad is None else _ld_any(residual_grad, "residual_grad", (rows, cols), (dY.dtype,))
        if out is None:
            out = torch.empty((rows, cols), dtype=dY.dtype, device=dY.device)
        lddx = _ld_any(out, "out", (rows, cols), (dY.dtype,))
        sums = torch.empty((2, cols), dtype=torch.float32, device=dY.device)
        t = _TYPE_OF_DTYPE[dY.dtype]
        nbytes = lib.layer_norm_backward_workspace_size(t, rows, cols)
        ws = launch.workspace(nbytes) if nbytes > 0 else None      # -1: the call itself names the error
        _check(lib.layer_norm_backward(
            t, rows, cols, dY.data_ptr(), lddy, X.data_ptr(), ldx, mean.data_ptr(), rstd.data_ptr(),
            2 if weight is None else _TYPE_OF_DTYPE[weight.dtype], _addr(weight), _addr(residual_grad), ldr,
            out.data_ptr(), lddx, sums.data_ptr(), sums.data_ptr() + 4 * cols, _addr(ws), max(nbytes, 0),
            launch.handle))
    return out, sums[0], sums[1]


# ---------------------------------------------------------- Newton-Schulz

NEWTON_SCHULZ_COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def newton_schulz(G, steps=5, coefficients=NEWTON_SCHULZ_COEFFICIENTS, eps=1e-7, out=None, stream=None):
    """The matrix G (2-D, or 3-D: a batch of matrices of one shape; bfloat16,
    float16 or float32) orthogonalised by ``steps`` Newton-Schulz steps of the
    odd polynomial with ``coefficients`` (a, b, c); see gemm_f32.h.  ``out``
    (G's shape and dtype) may be G."""
    with _Launch(stream, G, out) as launch:
        lib = load_library()
        if G.dim() not in (2, 3) or G.dtype not in _TYPE_OF_DTYPE:
            raise TypeError("G must be a 2-D or 3-D bfloat16, float16 or float32 tensor")
        if out is None:
            out = torch.empty(tuple(G.shape), dtype=G.dtype, device=G.device)
        elif out.shape != G.shape or out.dtype != G.dtype:
            raise ValueError("out must have G's shape and dtype")
        batch = G.shape[0] if G.dim() == 3 else 1
        rows, cols = G.shape[-2:]

        def strides(t, what):
            ld = _ld_any(t if t.dim() == 2 else t.as_strided(t.shape[1:], t.stride()[1:]), what)
            step = t.stride(0) if t.dim() == 3 and batch > 1 else max(rows - 1, 0) * ld + cols
            return ld, step

        ldg, stride_g = strides(G, "G")
        ldo, stride_o = strides(out, "out")
        t = _TYPE_OF_DTYPE[G.dtype]
        a, b, c = (float(v) for v in coefficients)
        nbytes = lib.newton_schulz_workspace_size(t, batch, rows, cols)
        ws = launch.workspace(nbytes) if nbytes > 0 else None      # -1: the call itself names the error
        _check(lib.newton_schulz(t, batch, rows, cols, G.data_ptr(), ldg, stride_g, int(steps), a, b, c, float(eps),
                                 out.data_ptr(), ldo, stride_o, _addr(ws), max(nbytes, 0), launch.handle))
    return out
