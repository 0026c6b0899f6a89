"""The 4-bit product at the ends of what its sums hold."""
from __future__ import annotations

import pytest
import torch

from gpu_support import say
from shared_memory_tiled_amd import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 16, 20, 50])
@pytest.mark.parametrize("group", [32, 64, 128, 256])
def test_large_finite_rows(M, group):
    """|x| = 2^116 throughout, every q and zero point, signs that cancel and signs
    that add: finite and right."""
    say(f"linear_w4 of 2^116: M={M} group={group}")
    N, K = 64, 512
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    q = torch.randint(0, 16, (N, K), generator=gen, device="cuda", dtype=torch.uint8)
    q[:8] = 15                                             # the largest sums
    z = torch.randint(-15, 16, (N, K // group), generator=gen, device="cuda")
    z[:4], z[4:8] = 15, -15
    scales = torch.full((N, K // group), 2.0 ** -20, dtype=torch.bfloat16, device="cuda")
    sign = torch.randint(0, 2, (M, K), generator=gen, device="cuda") * 2 - 1
    sign[0] = 1
    X = (sign * 2.0 ** 116).to(torch.bfloat16)
    y = binding.linear_w4(X, (q[:, 0::2] | q[:, 1::2] << 4).contiguous(), scales, zeros=z.to(torch.bfloat16),
                          group_size=group, out_dtype=torch.float32)
    # whole numbers times 2^96, a group's below 2^24: every sum is exact
    W = q.double() - z.double().repeat_interleave(group, 1)
    want = (sign.double() @ W.t().contiguous()) * 2.0 ** 96
    assert torch.equal(y.double(), want)
