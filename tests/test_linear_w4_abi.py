"""Refusals of the 4-bit layer's entry point, without a GPU."""
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


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


def call(lib, **kw):
    a = dict(fmt=0, M=8, N=16, K=200, A=FAKE, lda=200, Q=FAKE, ldq=100, group=64, scales=FAKE, lds=4, zeros=FAKE, ldz=4,
             C=FAKE, ldc=16)
    w = dict(ws=FAKE, ws_bytes=1 << 60)
    e = dict(c_type=0)
    for k, v in kw.items():
        (a if k in a else w if k in w else e)[k] = v
    return lib.gemm_w4_epilogue(*a.values(), ctypes.byref(binding.epilogue(**e)), w["ws"], w["ws_bytes"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(fmt=2), "INVALID_FORMAT"), (dict(c_type=1), "INVALID_TYPE"), (dict(activation=9), "INVALID_ACTIVATION"),
    (dict(gradient=1), "INVALID_EPILOGUE"), (dict(bias_grad=FAKE), "INVALID_EPILOGUE"),
    (dict(M=-1), "INVALID_DIM"), (dict(N=-1), "INVALID_DIM"), (dict(K=-1), "INVALID_DIM"),
    (dict(group=0), "INVALID_DIM"), (dict(group=16), "INVALID_DIM"), (dict(group=96), "INVALID_DIM"),
    (dict(group=-128), "INVALID_DIM"), (dict(group=192), "INVALID_DIM"),
    (dict(lda=199), "INVALID_LD"), (dict(ldq=99), "INVALID_LD"), (dict(lds=3), "INVALID_LD"), (dict(ldz=3), "INVALID_LD"),
    (dict(ldc=15), "INVALID_LD"), (dict(K=201, lda=201, ldq=100), "INVALID_LD"),
    (dict(residual=FAKE, ld_residual=15), "INVALID_LD"), (dict(residual=FAKE, ld_residual=17), "INVALID_LD"),
    (dict(A=None), "NULL_PTR"), (dict(Q=None), "NULL_PTR"), (dict(scales=None), "NULL_PTR"), (dict(C=None), "NULL_PTR"),
    (dict(A=FAKE + 1), "MISALIGNED"), (dict(scales=FAKE + 1), "MISALIGNED"), (dict(zeros=FAKE + 1), "MISALIGNED"),
    (dict(C=FAKE + 1), "MISALIGNED"), (dict(C=FAKE + 2, c_type=2), "MISALIGNED"),
    (dict(M=2 ** 31), "TOO_LARGE"), (dict(ldq=2 ** 62), "TOO_LARGE"), (dict(lds=2 ** 62), "TOO_LARGE"),
    (dict(group=2 ** 40), "TOO_LARGE"), (dict(N=2 ** 26, ldc=2 ** 26), "TOO_LARGE"), (dict(M=2 ** 22, N=1), "TOO_LARGE"),
    (dict(ws_bytes=-1), "INVALID_DIM"),
    (dict(M=0, A=None, C=None), "OK"), (dict(N=0, ldc=1, Q=None, scales=None, C=None), "OK"),
])
def test_refusals(lib, kw, want):
    assert call(lib, **kw) == CODES["GEMM_F32_OK" if want == "OK" else f"GEMM_F32_ERR_{want}"]


def test_workspace(lib):
    assert lib.gemm_w4_epilogue_workspace_size(1, 0, 64) == 0 and lib.gemm_w4_epilogue_workspace_size(0, 8, 64) == 0
    for bad in ((-1, 8, 64), (1, -8, 64), (1, 8, -64), (2 ** 22, 8, 64), (1, 2 ** 26, 64), (1, 8, 2 ** 31)):
        assert lib.gemm_w4_epilogue_workspace_size(*bad) == -1
    need = lib.gemm_w4_epilogue_workspace_size(40, 256, 16384)           # few columns, a long K
    assert need > 0 and need % (4 * 40 * 256) == 0
    big = dict(M=40, N=256, K=16384, lda=16384, ldq=8192, lds=256, ldz=256, ldc=256)
    assert call(lib, **big, ws_bytes=need - 1) == CODES["GEMM_F32_ERR_WORKSPACE"]
    assert call(lib, **big, ws=None) == CODES["GEMM_F32_ERR_NULL_PTR"]
    assert call(lib, **big, ws=FAKE + 4) == CODES["GEMM_F32_ERR_MISALIGNED"]


def test_binding_refuses_cpu_tensors():
    with pytest.raises(TypeError):
        binding.linear_w4(torch.zeros(1, 128, dtype=torch.bfloat16), torch.zeros(8, 64, dtype=torch.uint8),
                          torch.zeros(8, 1, dtype=torch.bfloat16))
