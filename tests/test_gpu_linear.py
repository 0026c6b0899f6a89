"""The product with its epilogue and its backward pass against binary64."""
from __future__ import annotations

import math

import pytest
import torch

import layer_refs as R
from gpu_support import say
from shared_memory_tiled_amd import binding

pytestmark = pytest.mark.gpu


def normal(seed, *shape, dtype=torch.bfloat16, scale=1.0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


def check_forward(M, N, K, dtype, kind, op_b="N", bias=True, residual=True, out_dtype=None, preact=True, seed=0,
                  op_a="N", strides=False, bias_dtype=None):
    say(f"linear M={M} N={N} K={K} {dtype} {kind} {op_a}{op_b} bias={bias} res={residual} out={out_dtype} "
        f"strides={strides}")
    X, W = normal(seed, M, K, dtype=dtype), normal(seed + 1, K, N, dtype=dtype, scale=max(K, 1) ** -0.5)
    b = normal(seed + 2, N, dtype=bias_dtype or dtype) if bias else None
    ot = out_dtype or dtype
    r = normal(seed + 3, M, N, dtype=ot) if residual else None
    Y, Z, S = R.linear_ref(X, W, b, kind, r)
    Xs = X.t().contiguous() if op_a == "T" else X
    Ws = W.t().contiguous() if op_b == "T" else W
    out, buf = None, None
    if strides:
        Xs, _ = R.padded(Xs, Xs.shape[1] + 3, 1)
        Ws, _ = R.padded(Ws, Ws.shape[1] + 5, 3)
        if r is not None:
            r, _ = R.padded(r, N + 7, 1)
        out, buf = R.padded(torch.zeros(M, N, dtype=ot, device="cuda"), N + 1, 5, fill=7.0)
    got = binding.linear(Xs, Ws, bias=b, activation=kind, residual=r, out=out, out_dtype=out_dtype,
                         return_preact=preact, op_a=op_a, op_b=op_b)
    y, z = got if preact else (got, None)
    torch.cuda.synchronize()
    R.within(y, Y, R.linear_tol(Y, Z, S, K, kind, None if r is None else r, ot), "out")
    if preact:
        R.within(z, Z, R.HALF[dtype] * Z.abs() + R.TINY[dtype] + (K + 2) * R.U * S, "preact")
    if buf is not None:
        R.untouched(buf, M, N, N + 1, 5)


@pytest.mark.parametrize("kind", R.ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("op_b", ["N", "T"])
def test_activations(kind, dtype, op_b):
    check_forward(70, 200, 136, R.DTYPES[dtype], kind, op_b)
    check_forward(5, 200, 136, R.DTYPES[dtype], kind, op_b)


# one token, decoding batches around the tile heights, odd sizes, sizes below
# every tile, one-value factors
SIZES = [(1, 64, 64), (1, 1, 1), (1, 1000, 4096), (2, 129, 8), (3, 7, 5), (8, 256, 8192), (15, 130, 96), (16, 128, 32),
         (17, 1000, 264), (31, 33, 4096), (32, 512, 1000), (33, 66, 40), (48, 4096, 136), (63, 65, 257), (64, 640, 1024),
         (3, 8200, 136), (40, 8192, 72), (5, 9, 300), (65, 320, 1024), (100, 100, 100), (127, 129, 131), (200, 1, 64), (257, 255, 1), (1000, 500, 24),
         (1000, 1002, 998), (999, 1001, 999), (2048, 200, 4096), (200, 190, 5000), (395, 72, 2132), (132, 414, 3923), (130, 130, 2050)]


@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("op_b", ["N", "T"])
def test_sizes(size, op_b):
    check_forward(*size, torch.bfloat16, "silu", op_b, seed=11)
    check_forward(*size, torch.float16, "none", op_b, residual=False, preact=False, out_dtype=torch.float32, seed=12)


@pytest.mark.parametrize("size", [(4, 130, 70), (30, 129, 257), (130, 258, 190), (700, 900, 72), (1100, 1300, 264)],
                         ids=str)
@pytest.mark.parametrize("op_a,op_b", [("N", "N"), ("N", "T"), ("T", "N"), ("T", "T")])
def test_strides_and_ops(size, op_a, op_b):
    check_forward(*size, torch.bfloat16, "gelu", op_b, op_a=op_a, strides=True, seed=21)
    check_forward(*size, torch.float16, "relu", op_b, op_a=op_a, seed=22, bias_dtype=torch.float32)


# every tile family once its count of tiles fits: 256, 192 and 160 tiles, the
# rows split between 256 and smaller ones, 128 and 64 tiles with K split
@pytest.mark.parametrize("size", [(2900, 2950, 130), (2300, 2310, 328), (4352, 4352, 64), (2048, 2040, 1032),
                                  (3000, 3300, 514), (1000, 1100, 2056), (4100, 4090, 70)], ids=str)
@pytest.mark.parametrize("op_b", ["N", "T"])
def test_large_tiles(size, op_b):
    check_forward(*size, torch.bfloat16, "gelu_tanh", op_b, seed=31)
    check_forward(*size, torch.float16, "silu", op_b, out_dtype=torch.float32, preact=False, seed=32)


def test_in_place_residual():
    for M, N, K in [(3, 200, 64), (50, 1000, 520), (300, 500, 264), (3000, 2900, 72), (33, 35, 37)]:
        X, W = normal(1, M, K), normal(2, K, N, scale=K ** -0.5)
        r = normal(3, M, N)
        Y, Z, S = R.linear_ref(X, W, None, "relu", r)
        out = r.clone()
        assert binding.linear(X, W, activation="relu", residual=out, out=out) is out
        R.within(out, Y, R.linear_tol(Y, Z, S, K, "relu", r, out.dtype), f"in place {M}x{N}x{K}")


def test_empty_and_no_inner():
    b = normal(5, 40)
    r = normal(6, 30, 40)
    X, W = torch.empty(30, 0, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 40, dtype=torch.bfloat16, device="cuda")
    y, z = binding.linear(X, W, bias=b, activation="silu", residual=r, return_preact=True)
    ref = R.act(b.double(), "silu") + r.double()
    R.within(y, ref, R.HALF[torch.bfloat16] * ref.abs() + 1e-6, "K = 0")
    assert torch.equal(z, b.expand(30, 40))
    assert binding.linear(normal(1, 0, 8), normal(2, 8, 4)).shape == (0, 4)
    assert binding.linear(normal(1, 4, 8), normal(2, 8, 0)).shape == (4, 0)
    d, db = binding.linear_grad(normal(1, 0, 8), normal(2, 16, 8), return_bias_grad=True)
    assert d.shape == (0, 16) and bool((db == 0).all())
    _, db = binding.activation_backward(normal(1, 0, 8))
    assert bool((db == 0).all())


def test_special_values():
    """Infinities and NaN stay in their rows and columns; NaN passes every
    activation; padding full of NaN reaches nothing."""
    for M, N, K in [(4, 64, 64), (40, 96, 64), (130, 130, 136), (700, 800, 72)]:
        for kind in R.ACTS:
            X, W = normal(1, M, K), normal(2, K, N, scale=K ** -0.5)
            X[1, 3] = float("nan")
            X[2, 5] = float("inf")
            y = binding.linear(X, W, activation=kind)
            assert bool(y[1].isnan().all()), (M, kind)
            rest = torch.cat([y[:1], y[3:]])
            assert bool(rest.isfinite().all()), (M, kind)
            pos = W[5] > 0
            assert bool((y[2][pos] == float("inf")).all())


def test_long_activation_range():
    """Preactivations from -60 to 60 and the types' extremes."""
    z = torch.cat([torch.linspace(-60, 60, 4001), torch.tensor([0.0, -0.0, 1e-30, -1e-30, 1e30, -1e30, 3e38, -3e38])])
    z = z.to(torch.float32).cuda()
    X = torch.zeros(z.numel(), 8, dtype=torch.bfloat16, device="cuda")
    W = torch.zeros(8, 4, dtype=torch.bfloat16, device="cuda")
    for kind in R.ACTS:
        res = None
        # the bias is the only term: one row of biases per call of 4009 columns
        y = binding.linear(X[:3], W[:, :1].expand(8, z.numel()).contiguous(), bias=z, activation=kind, residual=res,
                           out_dtype=torch.float32)
        ref = R.act(z.double(), kind).float().double()
        tol = 16 * R.U * ref.abs() + 16 * R.U * torch.exp(-z.double().abs() / 4) + 2.0 ** -126
        if kind in ("gelu_tanh", "silu"):      # the exponential's argument |x| costs |x| 2^-24 of a small tail
            x = z.double().abs() if kind == "silu" else 1.6 * (z.double().abs() + 0.044715 * z.double().abs() ** 3)
            tol = tol + ref.abs() * (x.clamp(max=200) + 4) * 2 * R.U
        if kind == "gelu":
            tol = tol + ref.abs() * ((z.double() ** 2).clamp(max=200) + 8) * 2 * R.U
        R.within(y[0], ref, tol, kind)


# ------------------------------------------------------------ backward pass

def grad_tol(D, V, Sv, K, Zd, kind, dtype):
    """Half a step of D; the binary32 sum's error times |act'| <= 1.13; the
    derivative's evaluation, within 32 units, times the sum."""
    return R.HALF[dtype] * D.abs() + R.TINY[dtype] + R.LIPSCHITZ * (K + 2) * R.U * Sv + \
        (32 * R.U * V.abs() if kind != "none" else 0.0)


@pytest.mark.parametrize("kind", R.ACTS)
@pytest.mark.parametrize("size", [(1, 40, 64), (20, 200, 136), (70, 200, 136), (333, 1000, 72), (999, 1001, 77),
                                  (2300, 2310, 264), (4100, 4090, 72), (130, 200, 3000)], ids=str)
def test_linear_grad(size, kind):
    M, N, K = size
    for dtype, out_dtype, residual in [(torch.bfloat16, None, False), (torch.float16, torch.float32, True)]:
        say(f"linear_grad {size} {kind} {dtype} residual={residual}")
        dZ, W, z = normal(1, M, K, dtype=dtype), normal(2, N, K, dtype=dtype, scale=K ** -0.5), normal(3, M, N, dtype=dtype)
        ot = out_dtype or dtype
        r = normal(4, M, N, dtype=ot) if residual else None
        V = dZ.double() @ W.double().t()
        Sv = dZ.double().abs() @ W.double().abs().t()
        if residual:
            V, Sv = V + r.double(), Sv + r.double().abs()
        D = V * R.act_derivative(z.double(), kind)
        tol = grad_tol(D, V, Sv, K, z, kind, ot)
        for op_b in ("T", "N"):
            Ws = W if op_b == "T" else W.t().contiguous()
            got, sums = binding.linear_grad(dZ, Ws, preact=z if kind != "none" else None, activation=kind, residual=r,
                                            out_dtype=out_dtype, return_bias_grad=True, op_b=op_b)
            R.within(got, D, tol, f"D {op_b}")
            # the sums add unrounded entries: their errors without the last rounding, and the sum's
            unrounded = tol - R.HALF[ot] * D.abs()
            R.within(sums, D.sum(0), unrounded.sum(0) + (M + 8) * R.U * D.abs().sum(0), f"sums {op_b}")


@pytest.mark.parametrize("kind", R.ACTS)
@pytest.mark.parametrize("size", [(1, 1), (1, 1000), (7, 33), (64, 129), (1000, 1001), (5000, 260), (16, 5000)], ids=str)
def test_activation_backward(size, kind):
    M, N = size
    for dtype in (torch.bfloat16, torch.float16):
        dY, z = normal(1, M, N, dtype=dtype), normal(2, M, N, dtype=dtype)
        dYp, _ = R.padded(dY, N + 3, 1)
        zp, _ = R.padded(z, N + 1, 3)
        D = dY.double() * R.act_derivative(z.double(), kind)
        dz, db = binding.activation_backward(dYp, zp if kind != "none" else None, kind)
        R.within(dz, D, R.HALF[dtype] * D.abs() + R.TINY[dtype] + 32 * R.U * dY.double().abs(), "dZ")
        tol = 32 * R.U * dY.double().abs().sum(0) + (M + 8) * R.U * D.abs().sum(0)
        R.within(db, D.sum(0), tol, "db")
        none, db2 = binding.activation_backward(dY, z if kind != "none" else None, kind, return_dz=False)
        assert none is None and torch.equal(db, db2)
        inplace = dY.clone()
        dz2, _ = binding.activation_backward(inplace, z if kind != "none" else None, kind, out=inplace,
                                             return_bias_grad=False)
        assert dz2 is inplace and torch.equal(dz2, dz)


@pytest.mark.parametrize("size", [(1, 64, 64), (64, 64, 64), (100, 72, 40), (999, 300, 130), (1001, 77, 501),
                                  (3001, 1000, 520), (2050, 2100, 2200), (8193, 128, 256)], ids=str)
@pytest.mark.parametrize("op_b", ["N", "T"])
def test_linear_backward(size, op_b):
    M, N, K = size
    for dtype, kind in ((torch.bfloat16, "gelu_tanh"), (torch.float16, "silu"), (torch.bfloat16, "none")):
        for wdt in (None, torch.float32):
            say(f"linear_backward {size} {op_b} {dtype} {kind} dW {wdt}")
            X, W = normal(1, M, K, dtype=dtype), normal(2, K, N, dtype=dtype, scale=K ** -0.5)
            dY, z = normal(3, M, N, dtype=dtype), normal(4, M, N, dtype=dtype)
            Ws = W.t().contiguous() if op_b == "T" else W
            dX, dW, db = binding.linear_backward(dY, X, Ws, preact=z if kind != "none" else None, activation=kind,
                                                 weight_grad_dtype=wdt, op_b=op_b)
            D = dY.double() * R.act_derivative(z.double(), kind)
            # dZ's own error: its rounding to dtype (none without an activation) and its evaluation
            ed = (R.HALF[dtype] * D.abs() + R.TINY[dtype] + 32 * R.U * dY.double().abs()) if kind != "none" else \
                torch.zeros_like(D)
            ref = D @ W.double().t()
            tol = R.HALF[dtype] * ref.abs() + R.TINY[dtype] + (ed + (N + 2) * R.U * D.abs()) @ W.double().abs().t() * 1.01
            R.within(dX, ref, tol, "dX")
            refw = X.double().t() @ D
            ot = wdt or dtype
            tolw = R.HALF[ot] * refw.abs() + R.TINY[ot] + X.double().abs().t() @ (ed + (M + 2) * R.U * D.abs()) * 1.01
            if op_b == "T":
                refw, tolw = refw.t(), tolw.t()
            R.within(dW, refw, tolw, "dW")
            tolb = 32 * R.U * dY.double().abs().sum(0) + (M + 8) * R.U * D.abs().sum(0)
            R.within(db, D.sum(0), tolb, "db")


def test_gradient_against_differences():
    """linear_backward against central differences of a binary64 loss."""
    M, N, K = 12, 20, 16
    X, W, dY = normal(1, M, K), normal(2, K, N, scale=0.3), normal(3, M, N)
    for kind in ("gelu", "gelu_tanh", "silu"):
        _, z = binding.linear(X, W, activation=kind, return_preact=True)
        dX, dW, db = binding.linear_backward(dY, X, W, preact=z, activation=kind)

        def loss(x, w, b):
            return (R.act(x @ w + b, kind) * dY.double()).sum()

        x, w, b = X.double(), W.double(), torch.zeros(N, dtype=torch.float64, device="cuda")
        h = 1e-5
        # the gradient is taken at Z rounded to bfloat16: |Z| 2^-8 |act''| of dY, and dZ's and the results' rounding
        slack = 3 * 2.0 ** -8
        for t, g, args in ((x, dX, 0), (w, dW, 1), (b, db, 2)):
            for idx in ([(0, 0), (3, 7), (11, 15)] if t.dim() == 2 and args == 0 else
                        [(0, 0), (5, 9), (15, 19)] if args == 1 else [(0,), (13,)]):
                p, m = t.clone(), t.clone()
                p[idx] += h
                m[idx] -= h
                a = [x, w, b]
                a[args] = p
                up = loss(*a)
                a[args] = m
                num = ((up - loss(*a)) / (2 * h)).item()
                zabs = (z.double().abs() * R.CURVATURE + R.LIPSCHITZ) * dY.double().abs()
                scale = (zabs @ w.abs().t())[idx] if args == 0 else (x.abs().t() @ zabs)[idx] if args == 1 else \
                    zabs.sum(0)[idx]
                assert abs(g[idx].item() - num) <= slack * scale.item() + 1e-6, (kind, args, idx, g[idx].item(), num)


def test_streams_and_graph_replay():
    """A captured layer, forward and backward, replayed between eager calls on
    other data gives the eager bits each time; two streams at once do not
    disturb each other."""
    for M, N, K in [(3, 512, 1024), (40, 640, 512), (200, 320, 264), (999, 333, 130)]:
        say(f"graph {M} {N} {K}")
        X, W, b = normal(1, M, K), normal(2, K, N, scale=K ** -0.5), normal(3, N)
        dY = normal(4, M, N)

        def layer():
            y, z = binding.linear(X, W, bias=b, activation="gelu", return_preact=True)
            return (y, z) + tuple(binding.linear_backward(dY, X, W, preact=z, activation="gelu"))

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            layer()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            captured = layer()
        for seed in range(3):
            X.copy_(normal(10 + seed, M, K))
            dY.copy_(normal(20 + seed, M, N))
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            kept = [t.clone() for t in captured]
            eager = layer()
            torch.cuda.synchronize()
            for a, e in zip(kept, eager):
                assert torch.equal(a, e)
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        torch.cuda.synchronize()
        outs = []
        for _ in range(4):
            outs.append(binding.linear(X, W, bias=b, activation="gelu", stream=s1))
            outs.append(binding.linear(X, W, bias=b, activation="gelu", stream=s2.cuda_stream))
        torch.cuda.synchronize()
        for o in outs:
            assert torch.equal(o, eager[0])


@pytest.mark.parametrize("kind", R.ACTS[1:])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_derivative_far_from_zero(kind, dtype):
    """Finite pre-activations of any size have a finite gradient: 0 or dY
    where the activation is flat or the identity."""
    far = [9.0, 29.0, 31.0, 100.0, 3000.0, 65504.0]
    if dtype is torch.bfloat16:
        far += [1e10, 1e13, 1e15, 1e19, 1e25, 3e38]
    z = torch.tensor([s * v for v in far for s in (1, -1)], device="cuda").to(dtype)[None, :].repeat(5, 1).contiguous()
    dY = normal(1, *z.shape, dtype=dtype)
    D = dY.double() * R.act_derivative(z.double(), kind)
    dz, _ = binding.activation_backward(dY, z, kind)
    R.within(dz, D, R.HALF[dtype] * D.abs() + R.TINY[dtype] + 32 * R.U * dY.double().abs(), kind)


@pytest.mark.parametrize("N,K", [(31, 256), (33, 600), (64, 2048), (1000, 1001), (2047, 513), (4097, 2048), (8192, 264),
                                 (4100, 2100)], ids=str)
@pytest.mark.parametrize("M", [1, 7, 16, 17, 32])
def test_few_rows_whole_depth(M, N, K):
    """Few rows whose blocks take all of K: ragged widths and depths, both
    storages, rows with a leading dimension, NaN beside them."""
    check_forward(M, N, K, torch.bfloat16, "silu", op_b="N")
    check_forward(M, N, K, torch.float16, "gelu", op_b="T", strides=True)
    check_forward(M, N, K, torch.bfloat16, "none", op_b="N", strides=True, out_dtype=torch.float32, preact=False)


@pytest.mark.parametrize("kind", R.ACTS)
def test_infinite_preactivations(kind):
    """Infinities take the limits: activation 0 and +inf, derivative 0 and 1
    (without one the product's entry itself); NaN stays NaN.  A binary16
    pre-activation past 65504 is such an infinity."""
    inf, nan = float("inf"), float("nan")
    one_sided = kind != "none"
    z = torch.tensor([inf, -inf, 2.0, inf, nan, -inf, 0.5, -1.0], device="cuda")
    # forward: the bias is the whole pre-activation; few rows, and tiles of every size
    for M, N, K in ((3, 8, 16), (70, 200, 32), (1000, 1100, 2056), (2900, 2952, 130)):
        say(f"{kind} forward {M} {N} {K}")
        b = z.repeat(-(-N // 8))[:N].contiguous()
        X, W = torch.zeros(M, K, dtype=torch.float16, device="cuda"), torch.zeros(K, N, dtype=torch.float16, device="cuda")
        y, kept = binding.linear(X, W, bias=b, activation=kind, out_dtype=torch.float32, return_preact=True)
        want = torch.where(b == -inf, torch.zeros_like(b) if one_sided else b, b)
        special = ~b.isfinite()
        for rows in (y[0], y[-1]):
            assert torch.equal(torch.nan_to_num(rows[special], nan=7.0, posinf=8.0, neginf=9.0),
                               torch.nan_to_num(want[special], nan=7.0, posinf=8.0, neginf=9.0))
            assert bool(rows[~special].isfinite().all())
        assert torch.equal(kept[0].isnan(), b.isnan()) and torch.equal(kept[0].abs() == inf, b.abs() == inf)
    for dtype in (torch.bfloat16, torch.float16):
        D = {-inf: 0.0 if one_sided else 1.0, inf: 1.0}
        for M, N, K in ((3, 40, 64), (70, 200, 72), (1000, 1096, 2056), (2900, 2952, 130)):
            say(f"{kind} gradient {M} {N} {K} {dtype}")
            zz = normal(5, M, N, dtype=dtype)
            zz[:, 3], zz[:, N - 1], zz[M - 1, 7], zz[M - 1, 8] = inf, -inf, inf, nan
            dY, W = normal(6, M, K, dtype=dtype), normal(7, N, K, dtype=dtype, scale=K ** -0.5)
            plain = binding.linear_grad(dY, W)                               # no activation
            d, sums = binding.linear_grad(dY, W, preact=zz, activation=kind, return_bias_grad=True)
            e, _ = binding.activation_backward(plain, zz, kind)
            for got in (d, e):
                for mask, factor in ((zz == inf, D[inf]), (zz == -inf, D[-inf])):
                    assert torch.equal(got[mask], plain[mask] * factor)
                assert torch.equal(got.isnan(), zz.isnan() if one_sided else torch.zeros_like(zz, dtype=torch.bool))
            assert torch.equal(sums.isnan(), d.isnan().any(0))


def test_preactivation_past_binary16():
    """Z near 10^5 keeps a finite binary32 result, an infinite binary16 Z and
    the gradient of the identity or of zero."""
    X = torch.full((33, 64), 40.0, dtype=torch.float16, device="cuda")
    W = torch.full((64, 72), 40.0, dtype=torch.float16, device="cuda")
    W[:, 1::2] = -40.0
    for kind in R.ACTS[1:]:
        y, z = binding.linear(X, W, activation=kind, out_dtype=torch.float32, return_preact=True)
        assert bool((y[:, ::2] == 102400.0).all()) and bool((y[:, 1::2] == 0).all()) and bool(z.isinf().all())
        dY = normal(1, 33, 72, dtype=torch.float16)
        dX, dW, db = binding.linear_backward(dY, X, W, preact=z, activation=kind)
        dZ, _ = binding.activation_backward(dY, z, kind)
        assert torch.equal(dZ[:, ::2], dY[:, ::2]) and bool((dZ[:, 1::2] == 0).all())
        assert bool(dX.isfinite().all()) and bool(dW.isfinite().all()) and bool(db.isfinite().all())


GRAD_SIZES = [(3, 200, 130), (40, 129, 257), (130, 258, 190), (300, 500, 264), (700, 1000, 72), (1000, 1100, 2056),
              (2900, 2951, 130), (2300, 2312, 264), (130, 200, 3001)]


@pytest.mark.parametrize("size", GRAD_SIZES, ids=str)
@pytest.mark.parametrize("op_a,op_b", [("N", "T"), ("N", "N"), ("T", "T"), ("T", "N")])
def test_linear_grad_strides_and_in_place(size, op_a, op_b):
    """Every argument with a leading dimension of its own, NaN beside the
    factors, pre-activation and residual, a frame around the output; and the
    residual's place as output."""
    M, N, K = size
    for dtype, ot, kind in ((torch.bfloat16, torch.bfloat16, "gelu"), (torch.float16, torch.float32, "silu")):
        say(f"linear_grad {size} {op_a}{op_b} {dtype} -> {ot} {kind}, strides")
        dZ, W = normal(1, M, K, dtype=dtype), normal(2, N, K, dtype=dtype, scale=K ** -0.5)
        z, r = normal(3, M, N, dtype=dtype), normal(4, M, N, dtype=ot)
        V = dZ.double() @ W.double().t() + r.double()
        Sv = dZ.double().abs() @ W.double().abs().t() + r.double().abs()
        D = V * R.act_derivative(z.double(), kind)
        tol = grad_tol(D, V, Sv, K, z, kind, ot)
        unrounded = tol - R.HALF[ot] * D.abs()
        sums_tol = unrounded.sum(0) + (M + 8) * R.U * D.abs().sum(0)
        dZs, Ws = (dZ.t().contiguous() if op_a == "T" else dZ), (W if op_b == "T" else W.t().contiguous())
        dZs, _ = R.padded(dZs, dZs.shape[1] + 3, 1)
        Ws, _ = R.padded(Ws, Ws.shape[1] + 5, 3)
        zs, _ = R.padded(z, N + 7, 3)
        rs, _ = R.padded(r, N + 2, 1)
        out, buf = R.padded(torch.zeros(M, N, dtype=ot, device="cuda"), N + 1, 5, fill=7.0)
        got, sums = binding.linear_grad(dZs, Ws, preact=zs, activation=kind, residual=rs, out=out, return_bias_grad=True,
                                        op_a=op_a, op_b=op_b)
        assert got is out
        R.within(out, D, tol, "D")
        R.within(sums, D.sum(0), sums_tol, "sums")
        R.untouched(buf, M, N, N + 1, 5)
        place, buf = R.padded(r, N + 3, 2, fill=7.0)
        got, sums2 = binding.linear_grad(dZs, Ws, preact=zs, activation=kind, residual=place, out=place,
                                         return_bias_grad=True, op_a=op_a, op_b=op_b)
        assert got is place and torch.equal(place, out) and torch.equal(sums, sums2)
        R.untouched(buf, M, N, N + 3, 2)


@pytest.mark.parametrize("size", [(3, 200, 130), (64, 64, 72), (1001, 77, 501), (999, 300, 130), (2050, 2100, 264),
                                  (8193, 128, 256)], ids=str)
@pytest.mark.parametrize("op_b", ["N", "T"])
def test_linear_backward_strides(size, op_b):
    """Arguments with leading dimensions of their own and NaN beside them: the
    bits of the contiguous call up to the order of sums, so within twice its
    tolerance of binary64 (checked there) -- here against binary64 itself."""
    M, N, K = size
    dtype, kind = torch.bfloat16, "gelu_tanh"
    say(f"linear_backward {size} {op_b}, strides")
    X, W = normal(1, M, K, dtype=dtype), normal(2, K, N, dtype=dtype, scale=K ** -0.5)
    dY, z = normal(3, M, N, dtype=dtype), normal(4, M, N, dtype=dtype)
    Xs, _ = R.padded(X, K + 3, 1)
    Ws, _ = R.padded(W.t().contiguous() if op_b == "T" else W, (K if op_b == "T" else N) + 5, 3)
    dYs, _ = R.padded(dY, N + 9, 1)
    zs, _ = R.padded(z, N + 1, 2)
    dX, dW, db = binding.linear_backward(dYs, Xs, Ws, preact=zs, activation=kind, op_b=op_b)
    D = dY.double() * R.act_derivative(z.double(), kind)
    ed = R.HALF[dtype] * D.abs() + 32 * R.U * dY.double().abs()
    ref = D @ W.double().t()
    tol = R.HALF[dtype] * ref.abs() + (ed + (N + 2) * R.U * D.abs()) @ W.double().abs().t() * 1.01
    R.within(dX, ref, tol, "dX")
    refw = X.double().t() @ D
    tolw = R.HALF[dtype] * refw.abs() + X.double().abs().t() @ (ed + (M + 2) * R.U * D.abs()) * 1.01
    if op_b == "T":
        refw, tolw = refw.t(), tolw.t()
    R.within(dW, refw, tolw, "dW")
    R.within(db, D.sum(0), 32 * R.U * dY.double().abs().sum(0) + (M + 8) * R.U * D.abs().sum(0), "db")


@pytest.mark.parametrize("size", [(256, 256, 8192), (130, 100, 5000), (129, 131, 8191), (500, 60, 4100), (72, 300, 6002)],
                         ids=str)
@pytest.mark.parametrize("op_a,op_b", [("T", "N"), ("N", "N"), ("N", "T"), ("T", "T")])
def test_few_tiles_and_a_long_depth(size, op_a, op_b):
    """K split over blocks: strides, odd sizes, the epilogue on the planes."""
    check_forward(*size, torch.bfloat16, "none", op_b, op_a=op_a, strides=True, bias=False, residual=False, preact=False)
    check_forward(*size, torch.float16, "silu", op_b, op_a=op_a, strides=True, seed=3)
    check_forward(*size, torch.bfloat16, "gelu", op_b, op_a=op_a, out_dtype=torch.float32, seed=5)


def test_small_tails_keep_their_relative_accuracy():
    """Activations of negative pre-activations far from zero, relative to their
    value, in units U = 2^-24 of it: the exponential is within 2 + 1.23 |x| at
    argument x (its unit's last place, the argument's scaling), reciprocals
    within 2, sums and products 1 each.
      silu       x = z: with 1 + e, reciprocal, product and store 5
      gelu       x = z^2 / 2, its own rounding 1 |x|; t and the polynomial 7e-7
                 (12 U), three products and the store 4.  The reference takes
                 erfc: torch's ndtr adds 1 to erf, in steps of 2^-54
      gelu_tanh  x = 2 u: four roundings of it 4 |x|; 5 as for silu"""
    z = torch.linspace(-12.0, -0.01, 6000, device="cuda")
    X, W = torch.zeros(3, 8, dtype=torch.bfloat16, device="cuda"), torch.zeros(8, z.numel(), dtype=torch.bfloat16, device="cuda")
    for kind, x, own, rest in (("silu", z, 0, 5), ("gelu", z * z / 2, 1, 12 + 4),
                               ("gelu_tanh", 1.6 * (z + 0.044715 * z ** 3), 4, 5)):
        y = binding.linear(X, W, bias=z, activation=kind, out_dtype=torch.float32)
        zd = z.double()
        ref = zd * 0.5 * torch.special.erfc(-zd / math.sqrt(2.0)) if kind == "gelu" else R.act(zd, kind)
        normal_range = ref.abs() > 2.0 ** -120
        tol = ref.abs() * (2 + rest + (1.23 + own) * x.double().abs()) * R.U
        R.within(y[1][normal_range], ref[normal_range], tol[normal_range], kind)
        assert bool((y[1][~normal_range].abs() <= 2.0 ** -119).all())


@pytest.mark.parametrize("size", [(1, 64, 64), (300, 200, 136), (1001, 77, 501)], ids=str)
def test_linear_backward_without_a_bias(size):
    """The same bits of dX and dW, no sums; also on another stream."""
    M, N, K = size
    X, W, dY, z = normal(1, M, K), normal(2, K, N, scale=K ** -0.5), normal(3, M, N), normal(4, M, N)
    for kind, pre in (("none", None), ("silu", z)):
        dX, dW, _ = binding.linear_backward(dY, X, W, preact=pre, activation=kind)
        torch.cuda.synchronize()
        for stream in (None, torch.cuda.Stream()):
            got = binding.linear_backward(dY, X, W, preact=pre, activation=kind, stream=stream, return_bias_grad=False)
            torch.cuda.synchronize()
            assert got[2] is None and torch.equal(got[0], dX) and torch.equal(got[1], dW)
