"""The layer over groups at sizes that take its widest tiles: more of them than
the chip holds at once, with a few left over, rows and columns that end inside
one, results that go past the caches."""
from __future__ import annotations

import pytest
import torch

import layer_refs as R
from gpu_support import say
from shared_memory_tiled_amd import binding
from test_gpu_grouped import check_backward, check_forward, normal

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


@pytest.mark.parametrize("M,N", [(3, (1 << 20) + 3), (70, 1 << 21), (1, 600001)], ids=str)
def test_activation_of_wide_rows(M, N):
    """More tiles side by side than a run of tiles down a group holds."""
    say(f"grouped activation of wide rows {M} {N}")
    dY, z = normal(1, M, N), normal(2, M, N)
    ends = [0, M // 2, M]
    dZ, db = binding.grouped_activation_backward(dY, torch.tensor(ends, dtype=torch.int32, device="cuda"), z, "silu")
    torch.cuda.synchronize()
    d = dY.double() * R.act_derivative(z.double(), "silu")
    R.within(dZ, d, R.HALF[dY.dtype] * d.abs() + 32 * R.U * dY.double().abs(), "dZ")
    for g, (a, e) in enumerate(zip(ends, ends[1:])):
        tol = 32 * R.U * dY[a:e].double().abs().sum(0) + (e - a + 8) * R.U * d[a:e].abs().sum(0)
        R.within(db[g], d[a:e].sum(0), tol, f"db of group {g}")


@pytest.mark.parametrize("M,ld", [(4500, 1 << 20), (1100, 1 << 22)], ids=str)
@pytest.mark.parametrize("op_b", ["N", "T"])
def test_far_apart(M, ld, op_b):
    """Rows and weights whose places pass 2^32 bytes and 2^32 elements."""
    say(f"grouped far apart {M} {ld} {op_b}")
    K, N, stride = 64, 72, (1 << 31) + 8
    cuts = [0, M // 3, M // 3 + 5, M]
    offsets = torch.tensor(cuts, dtype=torch.int32, device="cuda")

    def far(t):
        view = torch.empty(M * ld, dtype=t.dtype, device="cuda").view(M, ld)[:, :t.shape[1]]
        return view.copy_(t)

    X, W, dY = normal(1, M, K), normal(2, 3, K, N, scale=K ** -0.5), normal(3, M, N)
    Wd = W.transpose(1, 2).contiguous() if op_b == "T" else W
    Wf = torch.empty(2 * stride + K * N, dtype=W.dtype, device="cuda").as_strided(Wd.shape, (stride, Wd.shape[2], 1))
    Wf.copy_(Wd)
    Xf, dYf, out = far(X), far(dY), far(torch.zeros_like(dY))
    y = binding.grouped_linear(Xf, Wf, offsets, activation="silu", out=out, op_b=op_b)
    dX, dW, db = binding.grouped_linear_backward(dYf, Xf, Wf, offsets, preact=out, activation="silu", op_b=op_b)
    assert y is out
    dt = X.dtype
    for g, (a, e) in enumerate(zip(cuts, cuts[1:])):
        Y, Z, S = R.linear_ref(X[a:e], W[g], None, "silu", None)
        R.within(y[a:e], Y, R.linear_tol(Y, Z, S, K, "silu", None, dt), f"group {g}")
        d = dY[a:e].double() * R.act_derivative(out[a:e].double(), "silu")
        ed = R.HALF[dt] * d.abs() + 32 * R.U * dY[a:e].double().abs()
        Wg, Xg = W[g].double(), X[a:e].double()
        ref = d @ Wg.t().contiguous()
        tol = R.HALF[dt] * ref.abs() + (ed + (N + 2) * R.U * d.abs()) @ Wg.abs().t().contiguous() * 1.01
        R.within(dX[a:e], ref, tol, f"dX of group {g}")
        ref = Xg.t().contiguous() @ d
        tol = R.HALF[dt] * ref.abs() + Xg.abs().t().contiguous() @ (ed + (e - a + 2) * R.U * d.abs()) * 1.01
        R.within(dW[g].t() if op_b == "T" else dW[g], ref, tol, f"dW of group {g}")
        tol = 32 * R.U * dY[a:e].double().abs().sum(0) + (e - a + 8) * R.U * d.abs().sum(0)
        R.within(db[g], d.sum(0), tol, f"db of group {g}")


def uneven(M, groups):
    """M rows over groups of unequal sizes, one of them empty if there are several."""
    if groups == 1:
        return [M]
    weights = [1 + (5 * g) % 7 for g in range(groups)]
    weights[groups // 2] = 0
    counts = [M * w // sum(weights) for w in weights]
    counts[-1] += M - sum(counts)
    return counts


# rows, widths and depths at which the choice of tile and of the split of K changes
CHOICES = [(1, 300, 1000, 1000), (1, 300, 500, 2102), (1, 300, 166, 4096), (1, 1000, 2000, 1000), (1, 1000, 1000, 6432),
           (1, 1000, 2000, 4096), (1, 2000, 166, 8192), (1, 2000, 2000, 4096), (1, 4000, 1000, 6432),
           (1, 4000, 2000, 2102), (1, 4000, 2000, 4096), (1, 9000, 166, 4096), (1, 9000, 166, 6432), (1, 9000, 1000, 1000),
           (3, 300, 500, 2102), (3, 300, 166, 6432), (3, 300, 2000, 6432), (3, 2000, 1000, 4096), (3, 1000, 2000, 6432),
           (3, 2000, 2000, 6432), (3, 4000, 500, 4096), (3, 4000, 1000, 4096), (3, 4000, 2000, 6432), (3, 9000, 166, 4096),
           (22, 300, 500, 1000), (22, 300, 166, 8192), (22, 300, 2000, 2102), (22, 1000, 166, 6432), (22, 1000, 500, 4096),
           (22, 1000, 1000, 2102), (22, 1000, 2000, 4096), (22, 4000, 500, 6432), (22, 9189, 166, 6432),
           (22, 4000, 1000, 6432), (22, 4000, 2000, 1000), (22, 4000, 2000, 2102), (22, 9000, 2000, 1000)]


@pytest.mark.parametrize("case", CHOICES, ids=str)
@pytest.mark.parametrize("op_b", ["N", "T"])
def test_choices(case, op_b):
    groups, M, N, K = case
    check_forward(uneven(M, groups), N, K, torch.bfloat16, "none", op_b, residual=False, preact=False)
    check_forward(uneven(M, groups), N, K + 2, torch.float16, "gelu", op_b, lead=3, tail=1)


@pytest.mark.parametrize("case", [(1, 16384, 256, 256), (1, 9000, 512, 300), (2, 8000, 200, 304), (4, 8000, 1000, 1000),
                                  (3, 2000, 1000, 500), (22, 9189, 166, 500), (22, 9189, 500, 1000), (1, 4000, 2048, 3900),
                                  (6, 16384, 128, 640), (1, 700, 64, 64)], ids=str)
@pytest.mark.parametrize("op_b", ["N", "T"])
def test_gradient_choices(case, op_b):
    groups, M, N, K = case
    check_backward(uneven(M, groups), N, K, torch.bfloat16, "none", op_b)
    check_backward(uneven(M, groups), N, K, torch.float16, "silu", op_b, wdt=torch.float32, lead=1, tail=2)
