"""Refusals of the grouped layer's entry points, without a GPU."""
import ctypes
import os
import re

import pytest
import torch

from shared_memory_tiled_amd import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CODES = {m[0]: int(m[1]) for m in re.findall(r"#define\s+(GEMM_\w+)\s+(-?\d+)",
                                             open(os.path.join(ROOT, "include", "gemm_f32.h")).read())}
FAKE = 0x10000          # an aligned, never dereferenced address
BIG = 1 << 60


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


def code(name):
    return CODES["GEMM_F32_OK" if name == "OK" else f"GEMM_F32_ERR_{name}"]


def forward(lib, size_only=False, **kw):
    a = dict(op_b=0, fmt=0, groups=4, M=8, N=16, K=32, A=FAKE, lda=32, B=FAKE, ldb=16, stride_b=512, offsets=FAKE)
    t = dict(C=FAKE, ldc=16, ld_bias=16, ws=FAKE, ws_bytes=BIG)
    e = dict(c_type=0)
    for k, v in kw.items():
        (a if k in a else t if k in t else e)[k] = v
    ep = ctypes.byref(binding.epilogue(**e))
    if size_only:
        return lib.gemm_mixed_grouped_workspace_size(*a.values(), ep, t["ld_bias"])
    return lib.gemm_mixed_grouped(*a.values(), t["C"], t["ldc"], ep, t["ld_bias"], t["ws"], t["ws_bytes"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(op_b=2), "INVALID_OP"), (dict(fmt=2), "INVALID_FORMAT"), (dict(c_type=1), "INVALID_TYPE"),
    (dict(bias=FAKE, bias_type=1), "INVALID_TYPE"), (dict(activation=5), "INVALID_ACTIVATION"),
    (dict(gradient=1), "INVALID_EPILOGUE"), (dict(bias_grad=FAKE), "INVALID_EPILOGUE"),
    (dict(groups=-1), "INVALID_DIM"), (dict(M=-1), "INVALID_DIM"), (dict(N=-1), "INVALID_DIM"), (dict(K=-1), "INVALID_DIM"),
    (dict(lda=31), "INVALID_LD"), (dict(ldb=15), "INVALID_LD"), (dict(ldc=15), "INVALID_LD"),
    (dict(stride_b=-1), "INVALID_LD"), (dict(bias=FAKE, ld_bias=-1), "INVALID_LD"),
    (dict(residual=FAKE, ld_residual=15), "INVALID_LD"), (dict(preact=FAKE, ld_preact=15), "INVALID_LD"),
    (dict(residual=FAKE, ld_residual=17, C=FAKE), "INVALID_LD"),
    (dict(A=None), "NULL_PTR"), (dict(B=None), "NULL_PTR"), (dict(C=None), "NULL_PTR"), (dict(offsets=None), "NULL_PTR"),
    (dict(A=FAKE + 1), "MISALIGNED"), (dict(C=FAKE + 1), "MISALIGNED"), (dict(offsets=FAKE + 2), "MISALIGNED"),
    (dict(groups=65536), "TOO_LARGE"), (dict(M=2 ** 31), "TOO_LARGE"), (dict(stride_b=2 ** 62), "TOO_LARGE"),
    (dict(bias=FAKE, ld_bias=2 ** 62), "TOO_LARGE"),
    (dict(M=2 ** 20, N=2 ** 20, ldb=2 ** 20, ldc=2 ** 20, stride_b=2 ** 25), "TOO_LARGE"),
    (dict(ws_bytes=-1), "INVALID_DIM"),
    (dict(M=0, A=None, C=None), "OK"), (dict(N=0, ldb=1, ldc=1, B=None, C=None), "OK"),
    (dict(groups=0, offsets=None, B=None), "OK"),
])
def test_forward_refusals(lib, kw, want):
    assert forward(lib, **kw) == code(want)


def test_workspace_size_of_bad_arguments(lib):
    assert forward(lib, size_only=True, groups=-1) == -1
    assert forward(lib, size_only=True, gradient=1) == -1
    assert forward(lib, size_only=True) >= 0
    assert lib.activation_grad_grouped_workspace_size(-1, 4, 4) == -1
    assert lib.activation_grad_grouped_workspace_size(4, 2 ** 31, 4) == -1
    assert lib.activation_grad_grouped_workspace_size(65536, 4, 4) == -1
    assert lib.activation_grad_grouped_workspace_size(3, 0, 5) > 0       # the sums of no rows are written too


def grad(lib, **kw):
    a = dict(fmt=0, groups=4, rows=64, M=16, N=24, A=FAKE, lda=16, B=FAKE, ldb=24, offsets=FAKE, c_type=0, C=FAKE,
             ldc=24, stride_c=16 * 24, ws=FAKE, ws_bytes=BIG)
    a.update(kw)
    return lib.gemm_mixed_grouped_grad(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(fmt=-1), "INVALID_FORMAT"), (dict(c_type=1), "INVALID_TYPE"), (dict(groups=-1), "INVALID_DIM"),
    (dict(rows=-1), "INVALID_DIM"), (dict(M=-1), "INVALID_DIM"), (dict(N=-1), "INVALID_DIM"),
    (dict(lda=15), "INVALID_LD"), (dict(ldb=23), "INVALID_LD"), (dict(ldc=23), "INVALID_LD"),
    (dict(stride_c=16 * 24 - 1), "INVALID_LD"), (dict(stride_c=-5), "INVALID_LD"),
    (dict(A=None), "NULL_PTR"), (dict(B=None), "NULL_PTR"), (dict(C=None), "NULL_PTR"), (dict(offsets=None), "NULL_PTR"),
    (dict(A=FAKE + 1), "MISALIGNED"), (dict(C=FAKE + 2, c_type=2), "MISALIGNED"), (dict(offsets=FAKE + 1), "MISALIGNED"),
    (dict(groups=65536), "TOO_LARGE"), (dict(rows=2 ** 31), "TOO_LARGE"), (dict(lda=2 ** 62), "TOO_LARGE"),
    (dict(M=2 ** 20, N=2 ** 20, lda=2 ** 20, ldb=2 ** 20, ldc=2 ** 20, stride_c=2 ** 40), "TOO_LARGE"),
    (dict(ws_bytes=-1), "INVALID_DIM"),
    (dict(groups=0, offsets=None, C=None), "OK"), (dict(M=0, C=None), "OK"), (dict(N=0, ldb=1, ldc=1, C=None), "OK"),
])
def test_grad_refusals(lib, kw, want):
    assert grad(lib, **kw) == code(want)


def activation(lib, **kw):
    a = dict(act=1, fmt=0, groups=4, M=64, N=24, dY=FAKE, ldy=24, z=FAKE, ldz=24, offsets=FAKE, dZ=FAKE, lddz=24,
             sums=FAKE, ws=FAKE, ws_bytes=BIG)
    a.update(kw)
    return lib.activation_grad_grouped(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(fmt=2), "INVALID_FORMAT"), (dict(act=7), "INVALID_ACTIVATION"), (dict(M=-1), "INVALID_DIM"),
    (dict(groups=-1), "INVALID_DIM"), (dict(ldy=23), "INVALID_LD"), (dict(ldz=23), "INVALID_LD"),
    (dict(lddz=23), "INVALID_LD"), (dict(dZ=FAKE, lddz=25), "INVALID_LD"), (dict(dY=None), "NULL_PTR"),
    (dict(z=None), "NULL_PTR"), (dict(offsets=None), "NULL_PTR"), (dict(dY=FAKE + 1), "MISALIGNED"),
    (dict(sums=FAKE + 2), "MISALIGNED"), (dict(offsets=FAKE + 2), "MISALIGNED"), (dict(M=2 ** 31), "TOO_LARGE"),
    (dict(groups=65536), "TOO_LARGE"), (dict(ws_bytes=0), "WORKSPACE"), (dict(ws=None), "NULL_PTR"),
    (dict(ws=FAKE + 4), "MISALIGNED"), (dict(N=0, ldy=1, ldz=1, lddz=1), "OK"), (dict(dZ=None, sums=None), "OK"),
    (dict(groups=0, offsets=None), "OK"),
])
def test_activation_refusals(lib, kw, want):
    assert activation(lib, **kw) == code(want)


def test_binding_refuses_cpu_tensors():
    X, W = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(2, 8, 16, dtype=torch.bfloat16)
    o = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(TypeError):
        binding.grouped_linear(X, W, o)
    with pytest.raises(TypeError):
        binding.grouped_linear_backward(torch.zeros(4, 16, dtype=torch.bfloat16), X, W, o)
    with pytest.raises(TypeError):
        binding.grouped_activation_backward(torch.zeros(4, 16, dtype=torch.bfloat16), o)
