"""Newton-Schulz orthogonalisation against binary64.

The map is not contracting in every direction, so errors are bounded for
matrices whose small singular values are known: half a step of the entry plus
the errors of the products, relative to the result's root mean square.
"""
from __future__ import annotations

import math

import pytest
import torch

import layer_refs as R
from gpu_support import say
from shared_memory_tiled_amd import binding

pytestmark = pytest.mark.gpu


def momentum(seed, *shape, dtype=torch.float32, rank=8):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    strong = torch.randn(*shape[:-1], rank, generator=gen, device="cuda") @ \
        torch.randn(*shape[:-2], rank, shape[-1], generator=gen, device="cuda")
    return (1e-3 * (0.1 * strong + torch.randn(*shape, generator=gen, device="cuda"))).to(dtype)


def check(G, steps=5, coefficients=(3.4445, -4.7750, 2.0315), eps=1e-7, out=None):
    """Tolerance, relative to the largest singular value bound 1.3 spread over
    an entry (the result's root mean square r): a step multiplies a relative
    error of the factors by at most |a| + 2 |b| + 4 |c| = 21.1 in the worst
    alignment, but the errors of a product's factors are independent from
    entry to entry, so they enter as about their root mean square: per step
    |a| + |b| + |c| = 10.3 of it, five steps' errors meeting at once, and a
    maximum over 10^7 entries of six of them: 10.3 * sqrt(5) * 6 = 138
    root-mean-square roundings.  Factors kept to 2^-22 or better (binary32,
    binary16 results) have a root mean square rounding of 2^-23.8.  A
    product's binary32 sum of n terms adds its own: each addition rounds the
    partial sum by at most half a unit in the last place, 2^-23.5 / sqrt(12) =
    2^-25.3 of it in the root mean square, partial sum i of n terms of random
    sign has sqrt(i / n) of the final one's size, and the squares add up to
    n / 2: sqrt(n / 2) 2^-25.3 of the sum, n the longer side.  Factors
    rounded to 11 bits (bfloat16 results; 2^-12.8 with the diagonals kept
    apart in binary32) give 138 * 2^-12.8 < 2^-5.6."""
    step = 2.0 ** -23.8 + math.sqrt(max(G.shape[-2:]) / 2) * 2.0 ** -25.3
    got = binding.newton_schulz(G, steps=steps, coefficients=coefficients, eps=eps, out=out)
    torch.cuda.synchronize()
    ref = R.newton_schulz_ref(G, steps, coefficients, eps)
    assert bool(ref.isfinite().all())
    r = ref.square().mean((-1, -2), keepdim=True).sqrt()
    tol = R.HALF[G.dtype] * ref.abs() + R.TINY[G.dtype] + r * (2.0 ** -5.6 if G.dtype == torch.bfloat16 else 138 * step)
    R.within(got, ref, tol, f"{tuple(G.shape)} {G.dtype}")
    rms = ((got.double() - ref).square().mean((-1, -2)).sqrt() / r[..., 0, 0].clamp(min=1e-300)).max().item()
    say(f"newton_schulz {tuple(G.shape)} {G.dtype} steps={steps}: relative rms error {rms:.2e}")
    # and in the root mean square: the result's rounding and 10.3 sqrt(5) = 23 roundings of the factors
    bound = R.HALF[G.dtype] + 23 * (2.0 ** -12.8 if G.dtype == torch.bfloat16 else step)
    assert rms <= bound, (rms, bound)
    return got


SHAPES = [(1, 1), (1, 7), (9, 1), (2, 2), (16, 16), (17, 33), (63, 64), (64, 65), (100, 30), (31, 200), (128, 128),
          (130, 257), (300, 129), (500, 500), (257, 1000), (1000, 260), (640, 1300), (1030, 1025)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_shapes(shape, dtype):
    # binary16 holds 1e-3 values coarsely but exactly; the reference sees the same ones
    check(momentum(sum(shape), *shape, dtype=R.DTYPES[dtype]))


@pytest.mark.parametrize("shape", [(3, 40, 72), (2, 300, 200), (8, 128, 128), (5, 257, 513), (2, 1100, 700), (16, 65, 31),
                                   (3, 2000, 1000)], ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_batches(shape, dtype):
    G = momentum(1, *shape, dtype=R.DTYPES[dtype])
    got = check(G)
    one = binding.newton_schulz(G[1].contiguous())
    r = one.double().square().mean().sqrt()
    assert (one.double() - got[1].double()).abs().max() <= (2.0 ** -5 if dtype == "bf16" else 2.0 ** -14) * r


@pytest.mark.parametrize("shape", [(1800, 2000), (2304, 2304), (4096, 1100), (2700, 2800)], ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large(shape, dtype):
    check(momentum(3, *shape, dtype=R.DTYPES[dtype]))


def test_strides_and_in_place():
    for dt in (torch.bfloat16, torch.float32):
        G = momentum(5, 3, 150, 90, dtype=dt)
        want = binding.newton_schulz(G)
        buf = torch.full((3 * 160 * 101 + 64,), 7.0, dtype=dt, device="cuda")
        view = buf[3:3 + 3 * 160 * 101].view(3, 160, 101)[:, :150, :90]
        view.copy_(G)
        src = buf.clone()[3:3 + 3 * 160 * 101].view(3, 160, 101)[:, :150, :90]
        assert torch.equal(binding.newton_schulz(src), want)
        got = binding.newton_schulz(view, out=view)
        assert got is view and torch.equal(view, want)
        mask = torch.ones_like(buf, dtype=torch.bool)
        mask[3:3 + 3 * 160 * 101].view(3, 160, 101)[:, :150, :90] = False
        assert bool((buf[mask] == 7.0).all())


def test_steps_and_coefficients():
    G = momentum(7, 96, 160)
    for steps in (0, 1, 2, 8):
        check(G, steps=steps)
    check(G, steps=12, coefficients=(1.5, -0.5, 0.0))
    check(G, steps=6, coefficients=(1.875, -1.25, 0.375))
    check(G * 0, steps=5)
    check(G * 1e30, steps=5)
    check(G.float() * 1e-30, steps=5, eps=0.0)


def test_orthogonal_result():
    """After enough steps of a polynomial with a fixed point at 1, the rows
    are orthonormal to the precision of the factors."""
    for shape in ((96, 400), (400, 96)):
        X = binding.newton_schulz(momentum(9, *shape), steps=30, coefficients=(1.875, -1.25, 0.375)).double()
        S = X @ X.t() if shape[0] < shape[1] else X.t() @ X
        assert (S - torch.eye(96, dtype=torch.float64, device="cuda")).abs().max() <= 2.0 ** -18


def test_nan_stays_in_its_matrix():
    for dt in (torch.bfloat16, torch.float32):
        G = momentum(3, 4, 70, 130, dtype=dt)
        want = binding.newton_schulz(G)
        G[2, 3, 4] = float("nan")
        G[1, 69, 129] = float("inf")
        got = binding.newton_schulz(G)
        assert bool(got[2].isnan().all()) and bool(got[1].isnan().all())
        assert torch.equal(got[[0, 3]], want[[0, 3]])


def test_streams_and_graph_replay():
    for shape, dt in (((200, 300), torch.bfloat16), ((2, 520, 260), torch.float32), ((1024, 1024), torch.bfloat16)):
        G = momentum(1, *shape, dtype=dt)
        binding.newton_schulz(G)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            captured = binding.newton_schulz(G)
        for seed in range(3):
            G.copy_(momentum(10 + seed, *shape, dtype=dt))
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            kept = captured.clone()
            eager = binding.newton_schulz(G)
            torch.cuda.synchronize()
            assert torch.equal(kept, eager)
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        a = [binding.newton_schulz(G, stream=s) for s in (s1, s2, s1, s2)]
        torch.cuda.synchronize()
        assert all(torch.equal(t, eager) for t in a)
        assert math.isfinite(eager.float().sum().item())


@pytest.mark.parametrize("shape", [(0, 4, 6), (3, 0, 5), (3, 5, 0), (0, 7), (7, 0), (0, 0, 0)], ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_no_matrices(shape, dtype):
    G = torch.empty(shape, dtype=R.DTYPES[dtype], device="cuda")
    got = binding.newton_schulz(G)
    assert got.shape == G.shape and got.dtype == G.dtype
    assert binding.newton_schulz(G, out=G) is G


@pytest.mark.parametrize("shape", [(48, 80), (80, 48), (300, 500), (500, 300), (1000, 600), (600, 1000)], ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("by_row", [True, False])
def test_badly_scaled(shape, dtype, by_row):
    """Rows (columns) scaled over 1 .. 1e-9, judged row by row.

    Relative to its own row an entry has check()'s error.  To that comes what
    the planes cannot hold: half their last step, 2^-25 over a scale of 2^14, is
    q = 2^-39 of the norm, in the root mean square 2^-24 / 2^14 / sqrt(12) =
    2^-39.8.  An entry of X is off by it once for X itself and once for T, S and
    S S: those steps meet a column of X, whose norm is at most 1.3, with weights
    1, |b| = 4.8 and 2 |c| |S| = 2 * 2.03 * 1.7 = 6.9: together
    sqrt(1 + 1.3^2 (1 + 4.8^2 + 6.9^2)) = 11.1 of it per step.  The steps after
    it multiply an error by at most 3.4445 each, five steps' together by
    sqrt(sum of 3.4445^(2 j), j < 5) = 147.  Six root mean squares at the
    maximum: 6 * 147 * 11.1 * 2^-39.8 < 2^-26.5; a row's own root mean square
    error 147 * 11.1 * 2^-39.8 < 2^-29.1."""
    dt = R.DTYPES[dtype]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(sum(shape))
    n = shape[0] if by_row else shape[1]
    d = 10.0 ** (-9 * torch.arange(n, device="cuda") / (n - 1))
    G = (torch.randn(*shape, generator=gen, device="cuda") * (d[:, None] if by_row else d)).to(dt)
    got, ref = binding.newton_schulz(G).double(), R.newton_schulz_ref(G)
    if not by_row:
        got, ref = got.t(), ref.t()
    r = ref.square().mean(1, keepdim=True).sqrt()
    step = 2.0 ** -23.8 + math.sqrt(max(shape) / 2) * 2.0 ** -25.3
    rel = 2.0 ** -12.8 if dt == torch.bfloat16 else step
    R.within(got, ref, R.HALF[dt] * ref.abs() + 138 * rel * r + 2.0 ** -26.5, "entries")
    rms = (got - ref).square().mean(1).sqrt()
    R.within(rms, torch.zeros_like(rms), (R.HALF[dt] + 23 * rel) * r[:, 0] + 2.0 ** -29.1, "rows")


def test_below_the_planes():
    """Entries below half the planes' last step, 2^-39 of the norm, are 0;
    those above it have their polynomial's value: relative to it check()'s
    error, and the planes' 2^-39 at the start and after each step, which a
    further step multiplies by at most 3.4445."""
    for dt, rel in ((torch.float32, 138 * 2.0 ** -23.8), (torch.bfloat16, 2.0 ** -5.6)):
        values = [1.0, 2.0 ** -41, 2.0 ** -30, 2.0 ** -10]
        G = torch.zeros(70, 90, dtype=dt, device="cuda")
        for i, v in enumerate(values):
            G[i, i] = v
        got, ref = binding.newton_schulz(G, steps=3).double(), R.newton_schulz_ref(G, 3)
        assert got[1, 1].item() == 0
        assert got.count_nonzero().item() == 3
        floor = 2.0 ** -39 * sum(3.4445 ** k for k in range(4))
        for i in (0, 2, 3):
            error = (got[i, i] - ref[i, i]).abs().item()
            assert error <= (R.HALF[dt] + rel) * ref[i, i].item() + floor, (dt, values[i], error, ref[i, i].item())


def amplification(sigma, a, b, c, steps):
    """Per matrix, how much an error made before step k = 0 .. steps (after
    the last one for k = steps) counts in the result, to first order: in the
    basis of the singular vectors a step multiplies the parts of a change of X
    by the divided differences (p(s) - p(t)) / (s - t), (p(s) + p(t)) / (s + t) of
    its pairs of singular values (p'(s) for equal ones; t = 0 for the directions
    that only the longer side has)."""
    s = torch.cat([sigma, torch.zeros_like(sigma[..., :1])], -1)
    factors = []
    for _ in range(steps):
        x, y = s[..., :, None], s[..., None, :]
        xy, x2y2 = x * y, x * x + y * y
        # p over the pairs, the division done: s^3 and s^5's quotients
        minus = a + b * (x2y2 + xy) + c * (x ** 4 + x ** 3 * y + xy ** 2 + x * y ** 3 + y ** 4)
        plus = a + b * (x2y2 - xy) + c * (x ** 4 - x ** 3 * y + xy ** 2 - x * y ** 3 + y ** 4)
        factors.append(torch.stack([minus, plus]).abs())
        s = s * (a + s ** 2 * (b + c * s ** 2))
    after = [torch.ones_like(factors[0])]
    for f in reversed(factors):
        after.insert(0, f * after[0])
    return [t.amax((0, -1, -2)) for t in after]


@pytest.mark.parametrize("shape", [(1, 1), (1, 2), (2, 2), (3, 2), (3, 3), (4, 4), (2, 7), (8, 8), (16, 16), (17, 16),
                                   (32, 32), (64, 64)], ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_every_small_matrix(shape, dtype):
    """Thousands of small matrices, each within a bound of its own that holds
    for every one, not for most.  A product of factors of two planes is off by
    at most u of the product of their Frobenius norms: 2^-23 for what the planes
    of each factor do not hold and 2^-22 for the product of the low planes,
    2^-21 together, and 64 * 2^-24 = 2^-18 for the binary32 sum of up to 64 terms.
    With f = |X|_F a step then errs by 1.21 dT + u |T|_F f + 3.45 u f, where dS =
    u f^2 and dT = 4.775 dS + 2.04 (2 * 1.21^2 dS + u |S|_F^2); it counts in the
    result as amplification() says, and so does X_0's rounding, u f.  Half a
    step of the result is added."""
    a, b, c = binding.NEWTON_SCHULZ_COEFFICIENTS
    dt = R.DTYPES[dtype]
    n = 4096 if shape[0] <= 8 else 512
    gen = torch.Generator(device="cuda")
    gen.manual_seed(shape[0] * 100 + shape[1])
    G = (torch.randn(n, *shape, generator=gen, device="cuda") * 1e-2).to(dt)
    got, ref = binding.newton_schulz(G).double(), R.newton_schulz_ref(G)
    error, size = ((t).square().sum((-1, -2)).sqrt().cpu() for t in (got - ref, ref))
    sigma = torch.linalg.svdvals(G.double().cpu())
    sigma = sigma / (sigma.square().sum(-1, keepdim=True).sqrt() + 1e-7)
    u = 2.0 ** -21 + 2.0 ** -18
    counts = amplification(sigma, a, b, c, 5)
    total, s = u * counts[0], sigma
    for k in range(5):
        f, sf = s.square().sum(-1).sqrt(), (s ** 4).sum(-1).sqrt()
        tf = (b * s ** 2 + c * s ** 4).square().sum(-1).sqrt()
        ds = u * f ** 2
        dt_ = 4.775 * ds + 2.04 * (2 * 1.21 ** 2 * ds + u * sf ** 2)
        total = total + (1.21 * dt_ + u * tf * f + 3.45 * u * f) * counts[k + 1]
        s = (s * (a + s ** 2 * (b + c * s ** 2))).abs()
    bound = R.HALF[dt] * size + R.TINY[dt] * math.sqrt(shape[0] * shape[1]) + total
    say(f"{shape} {dtype}: largest relative error {(error / size).max().item():.1e}, of its bound {(error / bound).max().item():.2f}, "
        f"largest bound without the result's rounding {(total / size).max().item():.1e}")
    assert bool((error <= bound).all())
