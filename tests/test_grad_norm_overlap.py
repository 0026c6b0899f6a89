"""Where the norm of the gradients' clipping may lie: apart from what a call writes
and, written itself, from what it reads.  Without a GPU."""
import pytest

from shared_memory_tiled_amd import binding
from test_grad_norm_abi import FAKE, code, clip

A, B, OUT = FAKE + 0x1000, FAKE + 0x2000, (FAKE + 0x3000, FAKE + 0x4000)      # 16 binary32 values, 16 bfloat16 ones


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


@pytest.mark.parametrize("norm", [A, A + 4, A + 60, B, B + 28])
def test_norm_inside_a_gradient(lib, norm):
    # in place: written by some blocks while others read it
    assert clip(lib, grads=(A, B), norm=norm) == code("OVERLAP")
    assert clip(lib, grads=(A, B), norm=norm, both=False) == code("OVERLAP")
    # into other tensors: the call of both writes it while gradients are read; clipping alone only reads
    assert clip(lib, grads=(A, B), out=OUT, norm=norm) == code("OVERLAP")
    assert clip(lib, grads=(A, B), out=OUT, norm=norm, both=False) != code("OVERLAP")


@pytest.mark.parametrize("norm", [OUT[0], OUT[0] + 32, OUT[1] + 28])
def test_norm_inside_an_output(lib, norm):
    assert clip(lib, grads=(A, B), out=OUT, norm=norm) == code("OVERLAP")
    assert clip(lib, grads=(A, B), out=OUT, norm=norm, both=False) == code("OVERLAP")


@pytest.mark.parametrize("norm", [A - 4, A + 64, B - 4, B + 32, OUT[0] - 4, OUT[0] + 64, OUT[1] + 32])
def test_norm_beside_them(lib, norm):
    for out in (None, OUT):
        for both in (True, False):
            assert clip(lib, grads=(A, B), out=out, norm=norm, both=both) != code("OVERLAP")


@pytest.mark.parametrize("n", [255, 256, 257, 1000])
def test_norm_among_many(lib, n):
    grads = [FAKE + 0x100000 + 4096 * ((7 * i) % n) for i in range(n)]
    out = [p + 4096 * n for p in grads]
    kw = dict(grads=grads, sizes=[16] * n, types=[2] * n)
    for o, at in ((None, grads[n // 2]), (out, out[-1])):
        for both in (True, False):
            assert clip(lib, out=o, norm=at + 60, both=both, **kw) == code("OVERLAP")
            assert clip(lib, out=o, norm=at + 64, both=both, **kw) != code("OVERLAP")
    # an empty list or tensor has no place
    assert clip(lib, grads=(A, B), sizes=(0, 0), norm=A) != code("OVERLAP")
