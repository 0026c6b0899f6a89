"""Refusals of the gradients' norm and clipping, without a GPU."""
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


def arrays(grads, out, sizes, types):
    n = len(sizes)
    return (n, (ctypes.c_void_p * n)(*grads), (ctypes.c_void_p * n)(*out), (ctypes.c_int64 * n)(*sizes),
            (ctypes.c_int * n)(*types))


def clip(lib, grads=(FAKE, FAKE + 0x1000), out=None, sizes=(16, 16), types=(2, 0), max_norm=1.0, eps=1e-6, norm=FAKE,
         ws=FAKE, ws_bytes=BIG, both=True):
    n, g, o, s, t = arrays(grads, grads if out is None else out, sizes, types)
    if both:
        return lib.grad_clip_norm(n, g, o, s, t, max_norm, eps, norm, ws, ws_bytes, None)
    return lib.grad_clip(n, g, o, s, t, norm, max_norm, eps, None)


REFUSED = [
    (dict(sizes=(16, -1)), "INVALID_DIM"), (dict(sizes=(16, 2 ** 43)), "TOO_LARGE"), (dict(types=(2, 3)), "INVALID_TYPE"),
    (dict(types=(-1, 0)), "INVALID_TYPE"), (dict(grads=(None, FAKE)), "NULL_PTR"), (dict(grads=(FAKE, FAKE + 1)), "MISALIGNED"),
    (dict(grads=(FAKE + 2, FAKE + 0x1000)), "MISALIGNED"), (dict(out=(FAKE, None)), "NULL_PTR"),
    (dict(out=(FAKE + 2, FAKE + 0x1000)), "MISALIGNED"), (dict(norm=None), "NULL_PTR"), (dict(norm=FAKE + 2), "MISALIGNED"),
    (dict(max_norm=-1.0), "INVALID_SCALAR"), (dict(max_norm=float("nan")), "INVALID_SCALAR"),
    (dict(max_norm=float("inf")), "INVALID_SCALAR"), (dict(eps=0.0), "INVALID_SCALAR"), (dict(eps=float("nan")), "INVALID_SCALAR"),
    # the same tensor twice, an output inside another, over another's input, shifted over its own input
    (dict(grads=(FAKE, FAKE)), "OVERLAP"), (dict(grads=(FAKE, FAKE + 60)), "OVERLAP"),
    (dict(out=(FAKE + 0x1000, FAKE + 0x2000)), "OVERLAP"), (dict(out=(FAKE + 4, FAKE + 0x2000)), "OVERLAP"),
    (dict(out=(FAKE + 0x2000, FAKE + 0x2000 + 63)), "MISALIGNED"), (dict(out=(FAKE + 0x2000, FAKE + 0x2000 + 62)), "OVERLAP"),
    (dict(out=(FAKE + 0x1000, FAKE)), "OVERLAP"),
]


@pytest.mark.parametrize("kw,want", REFUSED)
def test_clip_refusals(lib, kw, want):
    assert clip(lib, **kw) == code(want)
    assert clip(lib, both=False, **kw) == code(want)


def test_many_tensors_and_overlap_at_the_end(lib):
    n = 1000
    grads = [FAKE + 4096 * ((7 * i) % n) for i in range(n)]
    grads[-1] = grads[3] + 32
    assert clip(lib, grads=grads, sizes=[16] * n, types=[2] * n) == code("OVERLAP")


def test_workspace(lib):
    n, g, o, s, t = arrays((FAKE, FAKE + 0x100000), (FAKE, FAKE + 0x100000), (100000, 5), (2, 0))
    need = lib.grad_norm_workspace_size(n, s)
    assert need > 0 and need % 8 == 0
    assert lib.grad_norm(n, g, s, t, FAKE, FAKE, need - 1, None) == code("WORKSPACE")
    assert lib.grad_norm(n, g, s, t, FAKE, None, need, None) == code("NULL_PTR")
    assert lib.grad_norm(n, g, s, t, FAKE, FAKE + 8, need, None) == code("MISALIGNED")
    assert lib.grad_norm(n, g, s, t, None, FAKE, need, None) == code("NULL_PTR")
    assert lib.grad_norm(-1, g, s, t, FAKE, FAKE, need, None) == code("INVALID_DIM")
    assert lib.grad_norm(n, None, s, t, FAKE, FAKE, need, None) == code("NULL_PTR")
    assert lib.grad_norm(n, g, None, t, FAKE, FAKE, need, None) == code("NULL_PTR")
    assert lib.grad_norm_workspace_size(-1, s) == -1 and lib.grad_norm_workspace_size(0, None) == 0
    assert lib.grad_norm_workspace_size(1, (ctypes.c_int64 * 1)(-4)) == -1


def test_binding_refuses():
    with pytest.raises(ValueError):
        binding.grad_norm([])
    with pytest.raises(TypeError):
        binding.grad_norm([torch.zeros(3)])
    with pytest.raises(TypeError):
        binding.clip_grad_norm([torch.zeros(3)], 1.0)
    assert binding.clip_grads([], None, 1.0) == []


@pytest.mark.parametrize("shape,stride,dense", [
    ((3, 4), (4, 1), True), ((3, 4), (1, 3), True), ((3, 4), (5, 1), False), ((2, 3, 4), (4, 8, 1), True),
    ((2, 3), (0, 1), False), ((3,), (2,), False), ((1, 3), (7, 1), True), ((4, 4), (2, 2), False),
])
def test_dense(shape, stride, dense):
    assert binding._dense(torch.empty(64).as_strided(shape, stride)) is dense


def test_lists_of_other_things():
    import torch

    t = torch.zeros(3)
    for bad in ([t], [None], [t, None], [3.0], ["x"]):
        with pytest.raises(TypeError):
            binding.grad_norm(bad)
        with pytest.raises(TypeError):
            binding.clip_grads(bad, t, 1.0)
        with pytest.raises(TypeError):
            binding.clip_grad_norm(bad, 1.0)
