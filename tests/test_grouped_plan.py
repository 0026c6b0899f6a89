"""The choice of tile and split of the grouped layer, on the host: no more blocks
along K than one round holds, for the kernel that the call takes."""
import ctypes
import random

import pytest

from host_code import compile_host

SOURCE = r"""
#include "grouped_plan.h"
using namespace gemmf32;
static void put(const Plan& q, int* out) {
    out[0] = q.direct;
    out[1] = q.bm;
    out[2] = q.bn;
    out[3] = q.splits;
}
extern "C" void plan(int groups, int rows, int N, int K, int op_b, int* out) {
    const int ldb = op_b ? K : N;
    const GroupedArgs a{groups, nullptr, rows, (int64_t)N * K, 0};
    put(make_plan(a, Gemm16Args{rows, N, K, nullptr, K, nullptr, ldb, nullptr, 0}, op_b), out);
}
extern "C" void grad_plan(int groups, int rows, int M, int N, int* out) {
    const GroupedArgs a{groups, nullptr, rows, (int64_t)M * N, 0};
    put(make_grad_plan(a, Gemm16Args{M, N, 0, nullptr, M, nullptr, N, nullptr, 0}), out);
}
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    return compile_host(tmp_path_factory.mktemp("plan"), SOURCE)


def plan(host, name, *args):
    out = (ctypes.c_int * 4)()
    getattr(host, name)(*args, out)
    return tuple(out)


# blocks on the chip: two to four on each of 256 CUs, as the kernels' registers and LDS leave
DIRECT = {(128, 256): 512, (128, 128): 768, (64, 256): 512, (64, 128): 768}
STAGED = [{(128, 128): 512, (64, 128): 1024}, {(128, 128): 768, (64, 128): 1024}]     # by op_b


def test_splits_of_gradients_fit_a_round(host):
    rng, split = random.Random(1), [0, 0]
    for _ in range(4000):
        groups, rows = rng.randint(1, 24), int(2 ** rng.uniform(6, 17))
        M, N = rng.randint(1, 2200), rng.randint(1, 2200)
        direct, bm, bn, splits = plan(host, "grad_plan", groups, rows, M, N)
        assert direct == (M % 2 == 0 and N % 2 == 0) and bm == 128
        if splits > 1:
            split[direct] += 1
            assert groups * -(-M // bm) * -(-N // bn) * splits <= (768 if direct else 512), (groups, rows, M, N, splits)
    assert min(split) > 100


def test_splits_of_layers_fit_a_round(host):
    rng, split = random.Random(2), [0, 0]
    for _ in range(4000):
        rows, op_b = int(2 ** rng.uniform(0, 14)), rng.randrange(2)
        N, K = rng.randint(1, 4200), int(2 ** rng.uniform(3, 14))
        direct, bm, bn, splits = plan(host, "plan", 1, rows, N, K, op_b)
        assert direct == (K % 2 == 0 and (op_b or N % 2 == 0))
        if splits > 1:
            split[direct] += 1
            slots = DIRECT if direct else STAGED[op_b]
            assert -(-rows // bm) * -(-N // bn) * splits <= slots[bm, bn], (rows, N, K, op_b, bm, bn, splits)
    assert min(split) > 100


# timed on both tiles, without a split
@pytest.mark.parametrize("rows,N,K,op_b,bm", [(4096, 2047, 4097, 0, 128), (4096, 2047, 4097, 1, 128), (8192, 4095, 2049, 0, 128),
                                              (8192, 4095, 1025, 1, 128), (2048, 2047, 4097, 1, 128), (1024, 1023, 1025, 1, 64)])
def test_the_faster_tile_of_odd_widths(host, rows, N, K, op_b, bm):
    assert plan(host, "plan", 1, rows, N, K, op_b)[1] == bm
