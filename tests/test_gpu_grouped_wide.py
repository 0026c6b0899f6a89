"""The layer over groups at sizes that take its widest tiles: more of them than
the chip holds at once, with a few left over, rows and columns that end inside
one, results that go past the caches."""
from __future__ import annotations

import pytest
import torch

from test_gpu_grouped import check_backward, check_forward

pytestmark = pytest.mark.gpu


# 595, 578 and 546 tiles of 128 x 256: the last 83, 66 and 34 in parts
@pytest.mark.parametrize("counts,N,K", [([4100, 200], 4104, 1544), ([1500, 900, 0, 1700], 4104, 2056),
                                        ([129, 1, 4990], 3200, 2102)], ids=["skewed", "4g", "short"])
@pytest.mark.parametrize("op_b", ["N", "T"])
def test_tiles_left_over(counts, N, K, op_b):
    check_forward(counts, N, K, torch.bfloat16, "gelu_tanh", op_b, residual=False)
    check_forward(counts, N, K, torch.float16, "silu", op_b, lead=1, tail=2, out_dtype=torch.float32)
    check_forward(counts, N, K, torch.float16, "relu", op_b, bias=False, preact=False, strides=True)


# weights' gradients of many tiles, of groups of few rows and of many; rows of whole lines, of 16 bytes, of neither
@pytest.mark.parametrize("counts,N,K", [([40] * 63 + [0], 512, 1024), ([3, 100, 0, 61] * 16, 520, 1000),
                                        ([33] * 70, 514, 998), ([50] * 65, 333, 1003), ([900, 0, 700], 2048, 4096),
                                        ([420, 380], 2056, 3600), ([385], 3850, 4090)],
                         ids=["lines", "runs", "even", "odd", "few", "few_runs", "one"])
@pytest.mark.parametrize("op_b", ["N", "T"])
def test_gradients_of_many_groups(counts, N, K, op_b):
    check_backward(counts, N, K, torch.bfloat16, "gelu_tanh", op_b)
    check_backward(counts, N, K, torch.float16, "none", op_b, wdt=torch.float32)
    check_backward(counts, N, K, torch.bfloat16, "none", op_b, strides=True)
