"""The size query of the weights' gradient with arguments out of range: -1, and no
sum or product that overflows on the way (compiled so that one ends the process)."""
import os
import subprocess
import sys

import pytest

from host_code import compile_host
from shared_memory_tiled_amd import binding

FAKE = 0x10000          # an aligned, never dereferenced address
SOURCE = r"""
#include "api_grouped.hip"
namespace gemmf32 {
int64_t grouped_workspace(const GroupedArgs&, const Gemm16Args&, int) { return 0; }
int64_t grouped_grad_workspace(const GroupedArgs&, const Gemm16Args&) { return 0; }
int64_t grouped_activation_workspace(int64_t, int64_t, int64_t) { return 0; }
hipError_t launch_grouped(const GroupedArgs&, const Gemm16Args&, const EpilogueArgs&, hipStream_t, int, int, void*) {
    return hipSuccess;
}
hipError_t launch_grouped_grad(const GroupedArgs&, const Gemm16Args&, const EpilogueArgs&, hipStream_t, int, void*) {
    return hipSuccess;
}
hipError_t launch_grouped_activation(const GroupedArgs&, const EpilogueArgs&, const uint16_t*, int64_t, float*,
                                     hipStream_t) {
    return hipSuccess;
}
}  // namespace gemmf32
"""
CALL = """
import ctypes, sys
lib = ctypes.CDLL(sys.argv[1])
q, i, p = lib.gemm_mixed_grouped_grad_workspace_size, ctypes.c_int64, ctypes.c_void_p
q.argtypes = [ctypes.c_int] + [i] * 4 + [p, i, p, i, p, ctypes.c_int]
q.restype = i
print(q(*map(int, sys.argv[2:])))
"""
BIG = 2 ** 63 - 1
# groups, rows, M, N, lda, ldb
REFUSED = [(4, 64, BIG, BIG, BIG, BIG), (4, 64, 2 ** 33, 2 ** 33, 2 ** 33, 2 ** 33), (4, 64, 2 ** 40, 16, 2 ** 40, 16),
           (4, 64, 16, 2 ** 62, 16, 2 ** 62), (4, BIG, 16, 16, 16, 16), (4, 2 ** 31, 16, 16, 16, 16),
           (4, 64, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31, 2 ** 31), (4, 64, -1, 16, 16, 16), (4, 64, 16, -1, 16, 16),
           (4, -1, 16, 16, 16, 16), (4, 64, -BIG, -BIG, 16, 16), (-1, 64, 16, 16, 16, 16), (65536, 64, 16, 16, 16, 16),
           (4, 64, 16, 16, 15, 16), (4, 64, 16, 16, 16, 15), (4, 64, 16, 16, BIG, 16)]


@pytest.fixture(scope="module")
def trapping(tmp_path_factory):
    path = tmp_path_factory.mktemp("trap")
    compile_host(path, SOURCE, "-ftrapv")
    return os.path.join(path, "host.so")


def arguments(groups, rows, M, N, lda, ldb):
    return 0, groups, rows, M, N, FAKE, lda, FAKE, ldb, FAKE, 0


@pytest.mark.parametrize("case", REFUSED, ids=str)
def test_refused_without_overflow(trapping, case):
    proc = subprocess.run([sys.executable, "-c", CALL, trapping, *map(str, arguments(*case))], capture_output=True, text=True)
    assert proc.returncode == 0 and int(proc.stdout) == -1, proc
    assert binding.load_library().gemm_mixed_grouped_grad_workspace_size(*arguments(*case)) == -1


@pytest.mark.parametrize("case", [(4, 64, 0, 16, 1, 16), (4, 64, 16, 0, 16, 1), (0, 64, 16, 16, 16, 16), (4, 0, 16, 16, 16, 16)])
def test_nothing_to_add(trapping, case):
    assert binding.load_library().gemm_mixed_grouped_grad_workspace_size(*arguments(*case)) == 0
