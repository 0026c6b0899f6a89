"""The weights' gradient of groups of about 2^31 rows."""
from __future__ import annotations

import pytest
import torch

from gpu_support import say
from shared_memory_tiled_amd import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("first,last", [(0, 2 ** 31 - 1), (5, 2 ** 31 - 700)], ids=str)
def test_gradient_of_a_long_group(first, last):
    """One column each: 32 blocks share the rows.  Whole numbers at the shares'
    ends and elsewhere, so that the sum is exact; NaN in rows of no group."""
    rows = 2 ** 31 - 1
    say(f"grouped gradient of rows {first} .. {last}")
    lib = binding.load_library()
    A = torch.zeros(rows, 1, dtype=torch.bfloat16, device="cuda")
    B = torch.ones(rows, 1, dtype=torch.bfloat16, device="cuda")
    share = (last - first + 1023) // 1024 * 32
    want = 0
    for i, at in enumerate([0, 1, 31, 2 ** 30 + 7, last - first - 1] +
                           [at for s in range(1, 32) for at in (s * share - 1, s * share)]):
        A[first + at, 0] = 1 + i
        B[first + at, 0] = 3
        want += 3 * (1 + i)
    A[:first], A[last:] = float("nan"), float("nan")
    offsets = torch.tensor([first, last], dtype=torch.int32, device="cuda")
    head = (0, 1, rows, 1, 1, A.data_ptr(), 1, B.data_ptr(), 1, offsets.data_ptr(), 2)
    need = lib.gemm_mixed_grouped_grad_workspace_size(*head)
    assert need == 4 * 32                              # a sum of each share
    ws = torch.full((need // 4,), float("nan"), device="cuda")
    C = torch.full((1,), float("nan"), device="cuda")
    status = lib.gemm_mixed_grouped_grad(*head, C.data_ptr(), 1, 1, ws.data_ptr(), need,
                                         torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert status == 0 and C.item() == want
