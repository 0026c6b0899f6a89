"""The order in which the weights' gradient adds a group's rows."""
from __future__ import annotations

import pytest
import torch

from gpu_support import say
from shared_memory_tiled_amd import binding
from test_gpu_grouped import normal, offsets_of

pytestmark = pytest.mark.gpu


# tiles of 128 columns; of 256 in two and in four rounds of 512
@pytest.mark.parametrize("rows,tiles,cols", [(4000, 3, 4), (700, 4, 5), (1100, 16, 16), (1000, 32, 16)], ids=str)
@pytest.mark.parametrize("op_b", ["N", "T"])
def test_the_same_in_every_tile(rows, tiles, cols, op_b):
    """Tiles of the same columns give the same bits wherever they lie: X's 256
    columns repeated, dY's likewise."""
    say(f"grouped gradient of repeated columns {rows} {tiles} {cols} {op_b}")
    X, dY = normal(1, rows, 256).repeat(1, tiles), normal(2, rows, 256).repeat(1, cols)
    K, N = X.shape[1], dY.shape[1]
    W = torch.zeros(2, *((N, K) if op_b == "T" else (K, N)), dtype=X.dtype, device="cuda")
    dW = binding.grouped_linear_backward(dY, X, W, offsets_of([rows - 100, 100])[1], op_b=op_b,
                                         weight_grad_dtype=torch.float32)[1]
    dW = dW.transpose(1, 2) if op_b == "T" else dW
    corner = dW[:, :256, :256]
    for i in range(tiles):
        for j in range(cols):
            assert torch.equal(dW[:, 256 * i:256 * (i + 1), 256 * j:256 * (j + 1)], corner), (i, j)
