"""Refusals of the layer operators' entry points, without a GPU."""
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


def test_constants_match_the_header():
    assert binding.TYPES == {"bf16": CODES["GEMM_MIXED_BF16"], "f16": CODES["GEMM_MIXED_F16"],
                             "f32": CODES["GEMM_MIXED_F32"]}
    for name, value in binding.ACTIVATIONS.items():
        assert CODES[f"GEMM_ACT_{name.upper()}"] == value
    # int32 x 4, then pointers and 64-bit values, in the header's order
    assert ctypes.sizeof(binding.Epilogue) == 4 * 4 + 6 * 8
    text = open(os.path.join(ROOT, "include", "gemm_f32.h")).read()
    body = text[text.index("typedef struct gemm_epilogue {"):text.index("} gemm_epilogue;")]
    names = re.findall(r"(\w+);\s*(?:/\*|\n)", body)
    assert names == [f[0] for f in binding.Epilogue._fields_]


def call(lib, ws=FAKE, ws_bytes=BIG, **kw):
    a = dict(op_a=0, op_b=0, fmt=0, M=8, N=16, K=32, A=FAKE, lda=32, B=FAKE, ldb=16, C=FAKE, ldc=16)
    e = dict(c_type=0)
    for k, v in kw.items():
        (a if k in a else e)[k] = v
    ep = binding.epilogue(**e)
    return lib.gemm_mixed_epilogue(a["op_a"], a["op_b"], a["fmt"], a["M"], a["N"], a["K"], a["A"], a["lda"], a["B"],
                                   a["ldb"], a["C"], a["ldc"], ctypes.byref(ep), ws, ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(op_a=2), "INVALID_OP"), (dict(op_b=-1), "INVALID_OP"),
    (dict(fmt=2), "INVALID_FORMAT"), (dict(fmt=-1), "INVALID_FORMAT"),
    (dict(c_type=1), "INVALID_TYPE"), (dict(c_type=3), "INVALID_TYPE"), (dict(c_type=-1), "INVALID_TYPE"),
    (dict(bias=FAKE, bias_type=1), "INVALID_TYPE"), (dict(bias=FAKE, bias_type=5), "INVALID_TYPE"),
    (dict(activation=5), "INVALID_ACTIVATION"), (dict(activation=-1), "INVALID_ACTIVATION"),
    (dict(gradient=2), "INVALID_EPILOGUE"), (dict(bias_grad=FAKE), "INVALID_EPILOGUE"),
    (dict(gradient=1, bias=FAKE), "INVALID_EPILOGUE"),
    (dict(M=-1), "INVALID_DIM"), (dict(N=-1), "INVALID_DIM"), (dict(K=-1), "INVALID_DIM"),
    (dict(lda=31), "INVALID_LD"), (dict(ldb=15), "INVALID_LD"), (dict(ldc=15), "INVALID_LD"),
    (dict(op_a=1, lda=7), "INVALID_LD"), (dict(op_b=1, ldb=31), "INVALID_LD"),
    (dict(residual=FAKE, ld_residual=15), "INVALID_LD"), (dict(preact=FAKE, ld_preact=0), "INVALID_LD"),
    (dict(gradient=1, activation=1, preact=FAKE, ld_preact=15), "INVALID_LD"),
    (dict(A=None), "NULL_PTR"), (dict(B=None), "NULL_PTR"), (dict(C=None), "NULL_PTR"),
    (dict(gradient=1, activation=1, ld_preact=16), "NULL_PTR"),
    (dict(A=FAKE + 1), "MISALIGNED"), (dict(B=FAKE + 1), "MISALIGNED"), (dict(C=FAKE + 1), "MISALIGNED"),
    (dict(C=FAKE + 2, c_type=2), "MISALIGNED"), (dict(bias=FAKE + 2, bias_type=2), "MISALIGNED"),
    (dict(residual=FAKE + 1, ld_residual=16), "MISALIGNED"), (dict(preact=FAKE + 1, ld_preact=16), "MISALIGNED"),
    (dict(gradient=1, bias_grad=FAKE + 2), "MISALIGNED"),
    (dict(M=2 ** 31), "TOO_LARGE"), (dict(K=2 ** 31, lda=2 ** 31), "TOO_LARGE"), (dict(lda=2 ** 62), "TOO_LARGE"),
    (dict(M=2 ** 30, N=2 ** 30, ldb=2 ** 30, ldc=2 ** 30), "TOO_LARGE"),
    (dict(M=0, A=None, C=None), "OK"), (dict(N=0, ldb=1, ldc=1, B=None, C=None), "OK"),
])
def test_epilogue_refusals(lib, kw, code):
    want = CODES["GEMM_F32_OK" if code == "OK" else f"GEMM_F32_ERR_{code}"]
    assert call(lib, **kw) == want


def test_epilogue_null_and_workspace(lib):
    head = (0, 0, 0, 8, 16, 32, FAKE, 32, FAKE, 16)
    assert lib.gemm_mixed_epilogue(*head, FAKE, 16, None, None, 0, None) == CODES["GEMM_F32_ERR_NULL_PTR"]
    # a product of operands past 2 GiB, with column sums: needs a workspace
    ep = binding.epilogue(0, gradient=1, bias_grad=FAKE)
    big = (0, 0, 0, 4096, 4096, 4096, FAKE, 1 << 20, FAKE, 4096)
    need = lib.gemm_mixed_epilogue_workspace_size(*big, ctypes.byref(ep))
    assert need > 0
    assert lib.gemm_mixed_epilogue(*big, FAKE, 4096, ctypes.byref(ep), FAKE, need - 1, None) == \
        CODES["GEMM_F32_ERR_WORKSPACE"]
    assert lib.gemm_mixed_epilogue(*big, FAKE, 4096, ctypes.byref(ep), None, need, None) == \
        CODES["GEMM_F32_ERR_NULL_PTR"]
    assert lib.gemm_mixed_epilogue(*big, FAKE, 4096, ctypes.byref(ep), FAKE + 4, need, None) == \
        CODES["GEMM_F32_ERR_MISALIGNED"]
    assert lib.gemm_mixed_epilogue(*big, FAKE, 4096, ctypes.byref(ep), FAKE, -1, None) == \
        CODES["GEMM_F32_ERR_INVALID_DIM"]
    assert lib.gemm_mixed_epilogue_workspace_size(0, 0, 0, -1, 4, 4, FAKE, 4, FAKE, 4, ctypes.byref(ep)) == -1


@pytest.mark.parametrize("args,code", [
    ((0, 2, 4, 8, FAKE, 8, FAKE, 8, FAKE, 8, FAKE), "INVALID_FORMAT"),
    ((9, 0, 4, 8, FAKE, 8, FAKE, 8, FAKE, 8, FAKE), "INVALID_ACTIVATION"),
    ((1, 0, -4, 8, FAKE, 8, FAKE, 8, FAKE, 8, FAKE), "INVALID_DIM"),
    ((1, 0, 4, 8, FAKE, 7, FAKE, 8, FAKE, 8, FAKE), "INVALID_LD"),
    ((1, 0, 4, 8, FAKE, 8, FAKE, 7, FAKE, 8, FAKE), "INVALID_LD"),
    ((1, 0, 4, 8, FAKE, 8, FAKE, 8, FAKE, 7, FAKE), "INVALID_LD"),
    ((1, 0, 4, 8, None, 8, FAKE, 8, FAKE, 8, FAKE), "NULL_PTR"),
    ((1, 0, 4, 8, FAKE, 8, None, 8, FAKE, 8, FAKE), "NULL_PTR"),
    ((1, 0, 4, 8, FAKE + 1, 8, FAKE, 8, FAKE, 8, FAKE), "MISALIGNED"),
    ((1, 0, 4, 8, FAKE, 8, FAKE, 8, FAKE, 8, FAKE + 2), "MISALIGNED"),
    ((1, 0, 2 ** 31, 8, FAKE, 8, FAKE, 8, FAKE, 8, FAKE), "TOO_LARGE"),
    ((0, 0, 4, 8, FAKE, 8, None, 0, None, 0, None), "OK"),
    ((1, 0, 0, 8, None, 8, None, 8, None, 8, None), "OK"),
])
def test_activation_grad_refusals(lib, args, code):
    want = CODES["GEMM_F32_OK" if code == "OK" else f"GEMM_F32_ERR_{code}"]
    assert lib.activation_grad(*args, FAKE, BIG, None) == want


def test_activation_grad_workspace(lib):
    need = lib.activation_grad_workspace_size(100, 300)
    assert need > 0 and lib.activation_grad_workspace_size(-1, 3) == -1
    args = (0, 0, 100, 300, FAKE, 300, None, 0, None, 0, FAKE)
    assert lib.activation_grad(*args, FAKE, need - 1, None) == CODES["GEMM_F32_ERR_WORKSPACE"]


def norm(lib, **kw):
    a = dict(type=0, rows=4, cols=8, x=FAKE, ldx=8, ptype=2, gamma=FAKE, beta=FAKE, eps=1e-5, y=FAKE, ldy=8,
             mean=FAKE, rstd=FAKE)
    a.update(kw)
    return lib.layer_norm(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(type=3), "INVALID_TYPE"), (dict(ptype=-1), "INVALID_TYPE"), (dict(rows=-1), "INVALID_DIM"),
    (dict(cols=0), "INVALID_DIM"), (dict(eps=-1e-3), "INVALID_SCALAR"), (dict(eps=float("nan")), "INVALID_SCALAR"),
    (dict(eps=float("inf")), "INVALID_SCALAR"), (dict(ldx=7), "INVALID_LD"), (dict(ldy=7), "INVALID_LD"),
    (dict(x=None), "NULL_PTR"), (dict(y=None), "NULL_PTR"), (dict(x=FAKE + 1), "MISALIGNED"),
    (dict(type=2, y=FAKE + 2), "MISALIGNED"), (dict(gamma=FAKE + 2), "MISALIGNED"), (dict(mean=FAKE + 1), "MISALIGNED"),
    (dict(rows=2 ** 31), "TOO_LARGE"), (dict(ldx=2 ** 62), "TOO_LARGE"), (dict(rows=0, x=None, y=None), "OK"),
])
def test_layer_norm_refusals(lib, kw, code):
    assert norm(lib, **kw) == CODES["GEMM_F32_OK" if code == "OK" else f"GEMM_F32_ERR_{code}"]


def norm_backward(lib, ws=FAKE, ws_bytes=BIG, **kw):
    a = dict(type=0, rows=4, cols=8, dy=FAKE, lddy=8, x=FAKE, ldx=8, mean=FAKE, rstd=FAKE, ptype=2, gamma=FAKE,
             r=FAKE, ldr=8, dx=FAKE, lddx=8, dgamma=FAKE, dbeta=FAKE)
    a.update(kw)
    return lib.layer_norm_backward(*a.values(), ws, ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(type=-1), "INVALID_TYPE"), (dict(ptype=4), "INVALID_TYPE"), (dict(rows=-2), "INVALID_DIM"),
    (dict(cols=0), "INVALID_DIM"), (dict(lddy=7), "INVALID_LD"), (dict(ldx=7), "INVALID_LD"),
    (dict(lddx=7), "INVALID_LD"), (dict(ldr=7), "INVALID_LD"), (dict(dy=None), "NULL_PTR"), (dict(x=None), "NULL_PTR"),
    (dict(mean=None), "NULL_PTR"), (dict(rstd=None), "NULL_PTR"), (dict(dx=None), "NULL_PTR"),
    (dict(dx=FAKE + 1), "MISALIGNED"), (dict(dgamma=FAKE + 2), "MISALIGNED"), (dict(r=FAKE + 1), "MISALIGNED"),
    (dict(rows=2 ** 31), "TOO_LARGE"), (dict(ws_bytes=0), "WORKSPACE"), (dict(ws=None), "NULL_PTR"),
    (dict(ws=FAKE + 4), "MISALIGNED"), (dict(ws_bytes=-5), "INVALID_DIM"),
    (dict(rows=0, dy=None, x=None, dgamma=None, dbeta=None), "OK"),
])
def test_layer_norm_backward_refusals(lib, kw, code):
    assert norm_backward(lib, **kw) == CODES["GEMM_F32_OK" if code == "OK" else f"GEMM_F32_ERR_{code}"]


def schulz(lib, ws=FAKE, ws_bytes=BIG, **kw):
    a = dict(type=0, batch=2, rows=4, cols=8, G=FAKE, ldg=8, sg=32, steps=5, a=3.4445, b=-4.775, c=2.0315, eps=1e-7,
             out=FAKE, ldo=8, so=32)
    a.update(kw)
    return lib.newton_schulz(*a.values(), ws, ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(type=3), "INVALID_TYPE"), (dict(batch=-1), "INVALID_DIM"), (dict(rows=-1), "INVALID_DIM"),
    (dict(cols=-1), "INVALID_DIM"), (dict(steps=-1), "INVALID_SCALAR"), (dict(steps=101), "INVALID_SCALAR"),
    (dict(a=float("nan")), "INVALID_SCALAR"), (dict(c=float("inf")), "INVALID_SCALAR"),
    (dict(a=1e4), "INVALID_SCALAR"), (dict(b=-1e30), "INVALID_SCALAR"), (dict(eps=-1.0), "INVALID_SCALAR"),
    (dict(ldg=7), "INVALID_LD"), (dict(ldo=7), "INVALID_LD"), (dict(sg=-1), "INVALID_LD"), (dict(so=31), "INVALID_LD"),
    (dict(batch=2 ** 31), "TOO_LARGE"), (dict(rows=2 ** 31), "TOO_LARGE"), (dict(sg=2 ** 62, batch=4), "TOO_LARGE"),
    (dict(G=None), "NULL_PTR"), (dict(out=None), "NULL_PTR"), (dict(G=FAKE + 1), "MISALIGNED"),
    (dict(type=2, out=FAKE + 2), "MISALIGNED"), (dict(ws_bytes=0), "WORKSPACE"), (dict(ws=None), "NULL_PTR"),
    (dict(ws=FAKE + 8), "MISALIGNED"), (dict(batch=0, G=None, out=None), "OK"), (dict(rows=0, so=0), "OK"),
])
def test_newton_schulz_refusals(lib, kw, code):
    assert schulz(lib, **kw) == CODES["GEMM_F32_OK" if code == "OK" else f"GEMM_F32_ERR_{code}"]


def test_size_queries(lib):
    assert lib.newton_schulz_workspace_size(0, 1, -1, 4) == -1 and lib.newton_schulz_workspace_size(5, 1, 4, 4) == -1
    assert lib.newton_schulz_workspace_size(0, 0, 4, 4) == 0 and lib.newton_schulz_workspace_size(0, 1, 64, 64) > 0
    assert lib.layer_norm_backward_workspace_size(0, 4, 0) == -1
    assert lib.layer_norm_backward_workspace_size(2, 4, 8) > 0


def test_tensor_forms_refuse_host_tensors():
    x = torch.zeros(4, 4, dtype=torch.bfloat16)
    for fn in (lambda: binding.linear(x, x), lambda: binding.linear_grad(x, x), lambda: binding.activation_backward(x),
               lambda: binding.linear_backward(x, x, x), lambda: binding.layer_norm(x),
               lambda: binding.newton_schulz(x)):
        with pytest.raises(TypeError):
            fn()


def test_activation_grad_column_limit(lib):
    """One block of 256 threads per 128 columns: the grid ends below 2^32."""
    n = 2 ** 31 - 64
    args = (0, 0, 1, n, FAKE, n, None, 0, None, 0, FAKE)
    assert lib.activation_grad_workspace_size(1, n) == -1
    assert lib.activation_grad(*args, FAKE, BIG, None) == CODES["GEMM_F32_ERR_TOO_LARGE"]


@pytest.mark.parametrize("M,N", [(2 ** 30, 2 ** 20), (2 ** 31 - 1, 2 ** 20), (2 ** 31 - 1, 2 ** 19), (2 ** 31 - 1, 2 ** 18),
                                 (2 ** 31 - 1, 2 ** 31 - 128), (1, 2 ** 31 - 128), (2 ** 31 - 1, 1), (1, 1), (9, 2 ** 31 - 128)])
def test_activation_grad_size_of_any_matrix(lib, M, N):
    """One partial row of N binary32 sums per block of rows; at most 2048
    blocks (and one more for the rest), at most one per 8 rows, and no fewer
    than one."""
    need = lib.activation_grad_workspace_size(M, N)
    assert 4 * N <= need <= 4 * N * min(2049, -(-M // 8)) + 256
    args = (0, 0, M, N, FAKE, N, None, 0, None, 0, FAKE)
    assert lib.activation_grad(*args, FAKE, need - 1, None) == CODES["GEMM_F32_ERR_WORKSPACE"]


@pytest.mark.parametrize("rows,cols", [(2 ** 31 - 1, 1), (1, 2 ** 31 - 1), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31 - 64, 2),
                                       (3 * 2 ** 29, 3 * 2 ** 29), (2 ** 30, 2 ** 30), (2 ** 16, 2 ** 16), (2 ** 23, 1)])
@pytest.mark.parametrize("batch", [1, 3])
def test_newton_schulz_matrices_past_the_limit(lib, batch, rows, cols):
    """Both planes of a matrix, padded to 64 and with 256 more rows and
    columns, have to stay below 2^31 bytes."""
    assert lib.newton_schulz_workspace_size(0, batch, rows, cols) == -1
    code = schulz(lib, batch=batch, rows=rows, cols=cols, ldg=cols, ldo=cols, sg=0, so=rows * cols)
    assert code == CODES["GEMM_F32_ERR_TOO_LARGE"]


def test_newton_schulz_matrices_up_to_the_limit(lib):
    for rows, cols in ((16384, 16384), (64, 2 ** 20), (1, 2 ** 20), (22848, 22848)):
        padded = -(-rows // 64) * 64 + 256, -(-cols // 64) * 64 + 256
        assert 4 * padded[0] * padded[1] < 2 ** 31
        assert lib.newton_schulz_workspace_size(2, 1, rows, cols) > 8 * rows * cols
    assert lib.newton_schulz_workspace_size(2, 65535, 64, 64) > 0
    assert lib.newton_schulz_workspace_size(2, 65536, 64, 64) == -1


def test_in_place_needs_the_same_leading_dimension(lib):
    """An output at an input's address with another leading dimension is
    another matrix over the same memory: refused; one row has none."""
    bad, ws = CODES["GEMM_F32_ERR_INVALID_LD"], CODES["GEMM_F32_ERR_WORKSPACE"]
    out = FAKE << 4
    assert call(lib, C=out, ldc=16, residual=out, ld_residual=24) == bad
    assert call(lib, C=out, ldc=24, residual=out, ld_residual=16, gradient=1) == bad
    # the next check is the workspace's, which a gradient of few rows needs
    assert call(lib, C=out, ldc=24, residual=out, ld_residual=24, gradient=1, ws_bytes=0) == ws
    assert call(lib, C=out, ldc=24, residual=out, ld_residual=16, gradient=1, M=1, ws_bytes=0) == ws
    grad = (0, 0, 4, 8, out, 8, None, 0, out, 9, FAKE)
    assert lib.activation_grad(*grad, FAKE, BIG, None) == bad
    assert lib.activation_grad(*grad[:9], 8, FAKE, FAKE, 0, None) == ws
    assert norm(lib, x=out, y=out, ldx=8, ldy=9) == bad
    assert norm(lib, x=out, y=out, ldx=10, ldy=9) == bad
    assert norm_backward(lib, dy=out, lddy=8, dx=out, lddx=9) == bad
    assert norm_backward(lib, r=out, ldr=12, dx=out, lddx=9) == bad
    assert norm_backward(lib, dy=out, lddy=9, dx=out, lddx=9, ws_bytes=0) == ws
    assert norm_backward(lib, r=out, ldr=12, dx=out, lddx=9, rows=1, ws_bytes=0) == ws


def test_layer_norm_backward_needs_no_workspace_without_sums(lib):
    """Past the workspace's check the call meets the missing device."""
    if torch.cuda.is_available():
        pytest.skip("the pointers are not memory: only where no kernel can start")
    bare = dict(dgamma=None, dbeta=None, ws=None, ws_bytes=0)
    assert norm_backward(lib, **bare) == CODES["GEMM_F32_ERR_DEVICE"]
    assert norm_backward(lib, **bare, rows=3, cols=40000, lddy=40000, ldx=40000, ldr=40000, lddx=40000) == \
        CODES["GEMM_F32_ERR_DEVICE"]
    for one in ("dgamma", "dbeta"):
        assert norm_backward(lib, **{**bare, one: FAKE}) == CODES["GEMM_F32_ERR_WORKSPACE"]
