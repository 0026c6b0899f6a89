"""Layer norm and its backward pass against binary64."""
from __future__ import annotations

import pytest
import torch

import layer_refs as R
from gpu_support import say
from shared_memory_tiled_amd import binding

pytestmark = pytest.mark.gpu

EPS = 1e-5
# one row, one column, both sides of every chunk and group width, long rows
SIZES = [(1, 1), (5, 1), (1, 2), (3, 7), (64, 8), (4, 63), (9, 64), (5, 65), (2, 511), (33, 512), (7, 513), (300, 1000),
         (1000, 1001), (17, 2047), (6, 2048), (3, 2050), (2, 4095), (70, 4096), (8, 4104), (5, 8192), (3, 8200),
         (2, 16384), (3, 16385), (2, 33000), (1, 70001), (3000, 24), (5003, 130), (2100, 768), (600, 5120), (40, 14336), (1030, 512)]


def make(seed, M, N, dtype, shift=0.5, scale=2.0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return (torch.randn(M, N, generator=gen, device="cuda") * scale + shift).to(dtype)


def forward_tols(x, w, b, y, mean, rstd, xhat, dtype):
    """mean: a tree sum of N terms, at most N / 64 + 20 additions deep; the
    deviations carry its error and a rounding; rstd half of the relative error
    of the variance and three roundings; y these, the scale and the shift."""
    N = x.shape[1]
    depth = N / 64 + 20
    xa = x.double().abs()
    e_mean = depth * R.U * xa.mean(1)
    dev = (x.double() - mean[:, None]).abs()
    # relative error of rstd: variance's sum (depth), its terms (2 roundings + 2 e_mean / sigma)
    e_rel = (depth / 2 + 6) * R.U + e_mean * rstd
    gamma = torch.ones(N, dtype=torch.float64, device=x.device) if w is None else w.double().abs()
    beta = torch.zeros_like(gamma) if b is None else b.double().abs()
    e_y = R.HALF[dtype] * y.abs() + R.TINY[dtype] + gamma * (xhat.abs() * (e_rel[:, None] + 4 * R.U) +
                                           (e_mean[:, None] + 2 * R.U * (dev + mean.abs()[:, None] * 0)) * rstd[:, None]) + \
        2 * R.U * (gamma * xhat.abs() + beta)
    return e_mean + R.U * mean.abs(), rstd * e_rel, e_y


@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_forward(size, dtype):
    M, N = size
    dt = R.DTYPES[dtype]
    for affine, strides in ((True, False), (False, True), (True, True)):
        say(f"layer_norm {size} {dtype} affine={affine} strides={strides}")
        x = make(1, M, N, dt)
        w = make(2, 1, N, torch.float32, 1.0, 0.2)[0] if affine else None
        b = make(3, 1, N, torch.float32, 0.0, 0.2)[0] if affine else None
        if affine and strides:
            w, b = w.to(dt), b.to(dt)
        xs, out, buf = x, None, None
        if strides:
            xs, _ = R.padded(x, N + 3, 1)
            out, buf = R.padded(torch.zeros_like(x), N + 1, 5, fill=7.0)
        y, mean, rstd = binding.layer_norm(xs, w, b, eps=EPS, out=out)
        ry, rmean, rrstd, xhat = R.layer_norm_ref(x, w, b, EPS)
        tm, tr, ty = forward_tols(x, w, b, ry, rmean, rrstd, xhat, dt)
        R.within(mean, rmean, tm, "mean")
        R.within(rstd, rrstd, tr, "rstd")
        R.within(y, ry, ty, "y")
        if buf is not None:
            R.untouched(buf, M, N, N + 1, 5)


def backward_ref(dy, x, mean, rstd, w, r):
    dyd, rs = dy.double(), rstd.double()[:, None]
    xhat = (x.double() - mean.double()[:, None]) * rs
    g = dyd * w.double() if w is not None else dyd
    n = x.shape[1]
    dx = rs * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    if r is not None:
        dx = dx + r.double()
    # rounding: each mean over N within depth units of its magnitudes (xhat's own 3 roundings, g's one)
    depth = n / 64 + 24
    e = rs * R.U * (4 * g.abs() + depth * g.abs().mean(1, keepdim=True) +
                    xhat.abs() * (depth + 8) * (g * xhat).abs().mean(1, keepdim=True) + 4 * g.abs())
    # x - mean rounds relative to the deviation only; nothing of |x| remains
    return dx, (dyd * xhat).sum(0), dyd.sum(0), e, (dyd * xhat).abs().sum(0), dyd.abs().sum(0)


@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_backward(size, dtype):
    M, N = size
    dt = R.DTYPES[dtype]
    for affine, residual, strides in ((True, False, False), (False, True, True), (True, True, True)):
        say(f"layer_norm_backward {size} {dtype} affine={affine} residual={residual} strides={strides}")
        x, dy = make(1, M, N, dt), make(2, M, N, dt, 0.05, 0.5)
        w = make(3, 1, N, torch.float32 if not strides else dt, 1.0, 0.2)[0] if affine else None
        r = make(4, M, N, dt, 0.0, 1.0) if residual else None
        _, mean, rstd, _ = R.layer_norm_ref(x, None, None, EPS)
        mean, rstd = mean.float(), rstd.float()
        xs, dys, rs_, out, buf = x, dy, r, None, None
        if strides:
            xs, _ = R.padded(x, N + 3, 1)
            dys, _ = R.padded(dy, N + 5, 3)
            if r is not None:
                rs_, _ = R.padded(r, N + 2, 1)
            out, buf = R.padded(torch.zeros_like(x), N + 1, 5, fill=7.0)
        dx, dw, db = binding.layer_norm_backward(dys, xs, mean, rstd, weight=w, residual_grad=rs_, out=out)
        rdx, rdw, rdb, e, sw, sb = backward_ref(dy, x, mean, rstd, w, r)
        tol = R.HALF[dt] * rdx.abs() + R.TINY[dt] + e + 2 * R.U * (0 if r is None else r.double().abs())
        R.within(dx, rdx, tol, "dx")
        R.within(dw, rdw, (M + 24) * R.U * sw, "dweight")
        R.within(db, rdb, (M + 16) * R.U * sb, "dbias")
        if buf is not None:
            R.untouched(buf, M, N, N + 1, 5)


def test_in_place_and_constant_rows():
    for dt in (torch.bfloat16, torch.float32):
        x = make(1, 37, 1000, dt)
        want = binding.layer_norm(x)[0]
        same = x.clone()
        assert binding.layer_norm(same, out=same)[0] is same and torch.equal(same, want)
        x[3] = 0.25
        y, mean, rstd = binding.layer_norm(x, eps=1e-2)
        assert bool((y[3] == 0).all()) and abs(rstd[3].item() - 10.0) < 1e-5 and mean[3].item() == 0.25
        dy = make(2, 37, 1000, dt)
        w = make(5, 1, 1000, torch.float32, 1.0, 0.1)[0]
        a = binding.layer_norm_backward(dy, x, mean, rstd, weight=w)
        g = dy.clone()
        b = binding.layer_norm_backward(g, x, mean, rstd, weight=w, out=g)
        assert b[0] is g and all(torch.equal(p, q) for p, q in zip(a, b))
        r = make(6, 37, 1000, dt)
        c = binding.layer_norm_backward(dy, x, mean, rstd, weight=w, residual_grad=r)[0]
        r2 = r.clone()
        assert torch.equal(binding.layer_norm_backward(dy, x, mean, rstd, weight=w, residual_grad=r2, out=r2)[0], c)


def test_large_mean():
    """A mean 4096 times the deviation: the two-pass variance keeps it (a
    one-pass one in binary32 would lose it)."""
    x = make(1, 9, 4000, torch.float32, 4096.0, 1.0)
    y, mean, rstd = binding.layer_norm(x, eps=EPS)
    ry, rmean, rrstd, xhat = R.layer_norm_ref(x, None, None, EPS)
    tm, tr, ty = forward_tols(x, None, None, ry, rmean, rrstd, xhat, torch.float32)
    R.within(mean, rmean, tm, "mean")
    R.within(rstd, rrstd, tr, "rstd")
    R.within(y, ry, ty, "y")


def test_special_values_stay_in_their_row():
    for N in (100, 4096, 70001):
        x = make(1, 6, N, torch.bfloat16)
        x[1, 2] = float("nan")
        x[4, 0] = float("inf")
        y = binding.layer_norm(x)[0]
        assert bool(y[1].isnan().all()) and bool(y[4].isnan().any())
        clean = binding.layer_norm(x[[0, 2, 3, 5]].contiguous())[0]
        assert torch.equal(y[[0, 2, 3, 5]], clean)


def test_no_rows():
    y, mean, rstd = binding.layer_norm(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"))
    assert y.shape == (0, 64) and mean.shape == (0,)
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    f = torch.empty(0, dtype=torch.float32, device="cuda")
    dx, dw, db = binding.layer_norm_backward(e, e, f, f)
    assert dx.shape == (0, 64) and bool((dw == 0).all()) and bool((db == 0).all())


def test_gradient_against_differences():
    M, N, h = 4, 48, 1e-5
    x, dy = make(1, M, N, torch.float32), make(2, M, N, torch.float32)
    w = make(3, 1, N, torch.float32, 1.0, 0.2)[0]
    _, mean, rstd = binding.layer_norm(x, w)
    dx, dw, db = binding.layer_norm_backward(dy, x, mean, rstd, weight=w)

    def loss(xx, ww, bb):
        return (R.layer_norm_ref(xx, ww, bb, EPS)[0] * dy.double()).sum()

    args = [x.double(), w.double(), torch.zeros(N, dtype=torch.float64, device="cuda")]
    for k, grad, indices in ((0, dx, [(0, 0), (2, 17), (3, 47)]), (1, dw, [(0,), (30,)]), (2, db, [(0,), (47,)])):
        for idx in indices:
            up, down = list(args), list(args)
            up[k], down[k] = args[k].clone(), args[k].clone()
            up[k][idx] += h
            down[k][idx] -= h
            num = ((loss(*up) - loss(*down)) / (2 * h)).item()
            # differences: h^2 and 2^-52 / h; the kernel: a few hundred units of terms of size 1
            assert abs(grad[idx].item() - num) <= 1e-5 * (1 + abs(num)), (k, idx, grad[idx].item(), num)


def test_graph_replay():
    for M, N, dt in ((8, 4096, torch.bfloat16), (1000, 768, torch.float32), (300, 9000, torch.float16)):
        x, dy, r = make(1, M, N, dt), make(2, M, N, dt), make(3, M, N, dt)
        w, b = make(4, 1, N, torch.float32, 1.0)[0], make(5, 1, N, torch.float32)[0]

        def both():
            y, mean, rstd = binding.layer_norm(x, w, b)
            return (y, mean, rstd) + binding.layer_norm_backward(dy, x, mean, rstd, weight=w, residual_grad=r)

        both()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            captured = both()
        for seed in range(3):
            x.copy_(make(10 + seed, M, N, dt))
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            kept = [t.clone() for t in captured]
            eager = both()
            torch.cuda.synchronize()
            assert all(torch.equal(a, e) for a, e in zip(kept, eager)), (M, N, seed)


def near_mean_tols(x, y, rstd, xhat, dtype):
    """For rows close to their mean: the first sum misses it by at most depth
    roundings of |x|, the deviations from that are exact (a subtraction of
    values within a factor of two), and their mean corrects the first one to
    depth roundings of the deviations."""
    N = x.shape[1]
    depth = N / 64 + 20
    xd = x.double()
    mean = xd.mean(1)
    first = depth * R.U * xd.abs().mean(1)
    left = depth * R.U * ((xd - mean[:, None]).abs().mean(1) + first)
    # relative error of the variance plus eps: sums and squares, and the shift that is left
    e_rel = (depth + 8) * R.U + (left * rstd) ** 2
    e_y = R.HALF[dtype] * y.abs() + xhat.abs() * (e_rel[:, None] + 6 * R.U) + (left * rstd)[:, None] * (1 + 4 * R.U)
    return left + R.U * mean.abs(), rstd * (e_rel + 3 * R.U), e_y


@pytest.mark.parametrize("N", [1, 3, 64, 1000, 1001, 4096, 4100, 8192, 10000, 16384, 33000, 70001])
def test_rows_of_one_value(N):
    """Every value equal: the mean is that value, y is zero but for what is
    left of the sums' roundings, though the sums themselves are not exact."""
    values = torch.tensor([0.1, 1000.3, 12345.678, -3.3e-5, 1.0 / 3.0, -7.7e4], device="cuda")
    for dt in (torch.float32, torch.float16, torch.bfloat16):
        c = values[values.abs() < (6e4 if dt == torch.float16 else 1e30)].to(dt)
        x = c[:, None].repeat(1, N).contiguous()
        y, mean, rstd = binding.layer_norm(x, eps=EPS)
        say(f"{N} {dt}: largest |y| {y.abs().max().item():.1e}")
        # depth roundings of depth roundings of the value, far below its own rounding
        left = ((N / 64 + 20) * R.U) ** 2 * c.double().abs()
        assert torch.equal(mean, c.float())
        R.within(y, torch.zeros_like(y), left[:, None] * EPS ** -0.5 * 1.01 + 1e-30, "y")
        R.within(rstd, torch.full_like(rstd, EPS ** -0.5), EPS ** -0.5 * (left ** 2 / EPS + 4 * R.U), "rstd")


@pytest.mark.parametrize("shift,scale", [(1e5, 1.0), (3e4, 0.05), (-7e6, 3.0), (100.0, 1e-4)])
@pytest.mark.parametrize("N", [100, 1001, 4096, 8192, 16384, 33000])
def test_rows_near_their_mean(N, shift, scale):
    """Means up to 10^6 deviations away, deviations down to a few units of the
    last place: y keeps the accuracy of the deviations."""
    x = make(N, 5, N, torch.float32, shift, scale)
    x[1] = shift
    x[1, N // 2] = torch.nextafter(x[1, N // 2], torch.tensor(float("inf"), device="cuda"))
    for eps in (1e-5, 1e-12):
        y, mean, rstd = binding.layer_norm(x, eps=eps)
        ry, rmean, rrstd, xhat = R.layer_norm_ref(x, None, None, float(torch.tensor(eps)))
        tm, tr, ty = near_mean_tols(x, ry, rrstd, xhat, torch.float32)
        R.within(mean, rmean, tm, "mean")
        R.within(rstd, rrstd, tr, "rstd")
        R.within(y, ry, ty, "y")


def test_backward_without_parameter_gradients():
    """dgamma and dbeta NULL: no workspace, the same dx bits."""
    lib = binding.load_library()
    for M, N, dt, t in ((5, 100, torch.bfloat16, 0), (300, 4096, torch.float16, 1), (7, 40000, torch.float32, 2)):
        x, dy = make(1, M, N, dt), make(2, M, N, dt)
        _, mean, rstd = binding.layer_norm(x)
        want = binding.layer_norm_backward(dy, x, mean, rstd)[0]
        dx = torch.empty_like(x)
        assert lib.layer_norm_backward(t, M, N, dy.data_ptr(), N, x.data_ptr(), N, mean.data_ptr(), rstd.data_ptr(), 2,
                                       None, None, 0, dx.data_ptr(), N, None, None, None, 0,
                                       torch.cuda.current_stream().cuda_stream) == 0
        assert torch.equal(dx, want)
        torch.cuda.synchronize()
        for stream in (None, torch.cuda.Stream()):
            got = binding.layer_norm_backward(dy, x, mean, rstd, stream=stream, return_param_grads=False)
            torch.cuda.synchronize()
            assert got[1] is None and got[2] is None and torch.equal(got[0], want)
