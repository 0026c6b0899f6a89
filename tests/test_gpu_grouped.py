"""The layer whose rows belong to groups with a weight each, and its backward
pass, against binary64: group by group from the definition."""
from __future__ import annotations

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


def offsets_of(counts, lead=0):
    ends = [lead]
    for c in counts:
        ends.append(ends[-1] + c)
    return ends, torch.tensor(ends, dtype=torch.int32, device="cuda")


def padded3(t, ld, gap, offset=0, fill=float("nan")):
    """A batch of matrices with row stride ld and `gap` elements between them."""
    groups, rows, cols = t.shape
    stride = rows * ld + gap
    buf = torch.full((offset + groups * stride + 64,), fill, dtype=t.dtype, device=t.device)
    view = buf[offset:].as_strided((groups, rows, cols), (stride, ld, 1), offset)
    view.copy_(t)
    return view


def check_forward(counts, N, K, dtype, kind, op_b="N", bias=True, residual=True, preact=True, out_dtype=None, lead=0,
                  tail=0, strides=False, bias_dtype=None, seed=0):
    say(f"grouped {counts if len(counts) < 20 else len(counts)} N={N} K={K} {dtype} {kind} {op_b} bias={bias} "
        f"res={residual} out={out_dtype} lead={lead} tail={tail} strides={strides}")
    ends, offsets = offsets_of(counts, lead)
    G, M = len(counts), ends[-1] + tail
    ot = out_dtype or dtype
    X = normal(seed, M, K, dtype=dtype)
    W = normal(seed + 1, G, K, N, dtype=dtype, scale=max(K, 1) ** -0.5)
    b = normal(seed + 2, G, N, dtype=bias_dtype or dtype) if bias else None
    r = normal(seed + 3, M, N, dtype=ot) if residual else None
    if M > ends[-1]:
        X[ends[-1]:] = float("nan")
    X[:lead] = float("nan")
    Xs, Ws, bs, rs = X, W.transpose(1, 2).contiguous() if op_b == "T" else W, b, r
    ldo, off = N, 0
    if strides:
        Xs, _ = R.padded(X, K + 3, 1)
        Ws = padded3(Ws, Ws.shape[2] + 5, 7, 3)
        ldo, off = N + 1, 5
        if r is not None:
            rs, _ = R.padded(r, N + 7, 1)
        if b is not None:
            bs, _ = R.padded(b, N + 3, 1)
    out, buf = R.padded(torch.full((M, N), 7.0, dtype=ot, device="cuda"), ldo, off, fill=7.0)
    got = binding.grouped_linear(Xs, Ws, offsets, bias=bs, activation=kind, residual=rs, out=out, return_preact=preact,
                                 op_b=op_b)
    y, z = got if preact else (got, None)
    torch.cuda.synchronize()
    for g, (s, e) in enumerate(zip(ends, ends[1:])):
        if s == e:
            continue
        rg = r[s:e] if residual else None
        Y, Z, S = R.linear_ref(X[s:e], W[g], b[g] if bias else None, kind, rg)
        R.within(y[s:e], Y, R.linear_tol(Y, Z, S, K, kind, rg, ot), f"out of group {g}")
        if preact:
            R.within(z[s:e], Z, R.HALF[dtype] * Z.abs() + R.TINY[dtype] + (K + 2) * R.U * S, f"preact of group {g}")
    mask = torch.ones(buf.numel(), dtype=torch.bool, device="cuda")     # rows of no group, and around the window
    for s, e in zip(ends, ends[1:]):
        mask[off + s * ldo:off + e * ldo].view(-1, ldo)[:, :N] = False
    assert bool((buf[mask] == 7.0).all()), "values of no group's row were written"


COUNTS = [[1], [0, 0, 3, 0], [5, 0, 64, 1], [16] * 16, [1, 2, 0, 3, 1] * 20, [130, 7, 0, 127, 129], [300, 700], [33],
          [0, 0], [1] * 70, [257, 0, 255, 1, 256]]


@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}g{sum(c)}r")
@pytest.mark.parametrize("op_b", ["N", "T"])
def test_counts(counts, op_b):
    check_forward(counts, 136, 72, torch.bfloat16, "silu", op_b, lead=3, tail=5)
    check_forward(counts, 129, 101, torch.float16, "none", op_b, residual=False, preact=False,
                  out_dtype=torch.float32, tail=64)


@pytest.mark.parametrize("N,K", [(1, 1), (64, 64), (7, 33), (1000, 8), (8, 1000), (257, 258), (520, 2056), (66, 1002),
                                 (1030, 130)])
@pytest.mark.parametrize("op_b", ["N", "T"])
def test_sizes(N, K, op_b):
    for counts in ([3, 0, 14, 1], [40, 200, 0, 90]):
        check_forward(counts, N, K, torch.bfloat16, "gelu", op_b)
        check_forward(counts, N, K, torch.float16, "relu", op_b, bias_dtype=torch.float32, seed=7)


@pytest.mark.parametrize("kind", R.ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_activations(kind, dtype):
    check_forward([3, 1], 200, 136, R.DTYPES[dtype], kind, "T")
    check_forward([70, 0, 300], 200, 136, R.DTYPES[dtype], kind)


@pytest.mark.parametrize("counts", [[2, 3, 1], [30, 20], [200, 0, 500, 131]], ids=str)
@pytest.mark.parametrize("op_b", ["N", "T"])
def test_strides(counts, op_b):
    check_forward(counts, 130, 70, torch.bfloat16, "gelu", op_b, strides=True, lead=2, tail=3)
    check_forward(counts, 256, 264, torch.float16, "gelu_tanh", op_b, strides=True, out_dtype=torch.float32)


# rows and weights enough for every kernel: large tiles, many small groups
@pytest.mark.parametrize("counts,N,K", [([1500, 900, 0, 1700], 2048, 520), ([2048, 2048], 2056, 264),
                                        ([70] * 60, 1024, 512), ([3000], 3000, 130), ([4100, 1, 90], 1290, 328)],
                         ids=["4g", "even", "many", "one", "skewed"])
@pytest.mark.parametrize("op_b", ["N", "T"])
def test_large(counts, N, K, op_b):
    check_forward(counts, N, K, torch.bfloat16, "gelu_tanh", op_b, residual=False)
    check_forward(counts, N, K, torch.float16, "silu", op_b, bias=False, preact=False, out_dtype=torch.float32)


def test_empty():
    X, W = normal(1, 6, 8), normal(2, 3, 8, 16)
    offsets = offsets_of([2, 0, 4])[1]
    assert binding.grouped_linear(X[:0], W, torch.zeros(4, dtype=torch.int32, device="cuda")).shape == (0, 16)
    out = torch.full((6, 16), 7.0, dtype=torch.bfloat16, device="cuda")
    binding.grouped_linear(X, W[:0], torch.zeros(1, dtype=torch.int32, device="cuda"), out=out)
    binding.grouped_linear(X, W, torch.full((4,), 3, dtype=torch.int32, device="cuda"), out=out)
    assert bool((out == 7.0).all())
    assert binding.grouped_linear(X, W[:, :, :0], offsets).shape == (6, 0)
    b = normal(5, 3, 16)
    y = binding.grouped_linear(X[:, :0], W[:, :0], offsets, bias=b, activation="silu")
    ref = R.act(b.double(), "silu")[torch.tensor([0, 0, 2, 2, 2, 2], device="cuda")]
    R.within(y, ref, R.HALF[torch.bfloat16] * ref.abs() + 1e-6, "K = 0")
    for wdt in (None, torch.float32):
        dX, dW, db = binding.grouped_linear_backward(normal(3, 0, 16), X[:0], W, torch.zeros_like(offsets),
                                                     weight_grad_dtype=wdt)
        assert dX.shape == (0, 8) and bool((dW == 0).all()) and bool((db == 0).all())


def test_shared_weight_and_bias():
    """Weights and biases broadcast over the groups (stride 0)."""
    X, W, b = normal(1, 300, 136), normal(2, 136, 200, scale=0.1), normal(3, 200)
    offsets = offsets_of([100, 7, 193])[1]
    y = binding.grouped_linear(X, W.expand(3, 136, 200), offsets, bias=b.expand(3, 200), activation="silu")
    Y, Z, S = R.linear_ref(X, W, b, "silu", None)
    R.within(y, Y, R.linear_tol(Y, Z, S, 136, "silu", None, y.dtype), "shared")


def test_in_place_residual_and_special_values():
    for counts in ([2, 3], [100, 29]):
        ends, offsets = offsets_of(counts)
        M = ends[-1]
        X, W, r = normal(1, M, 64), normal(2, 2, 64, 72, scale=0.1), normal(3, M, 72)
        out = r.clone()
        assert binding.grouped_linear(X, W, offsets, residual=out, out=out) is out
        for g in range(2):
            s, e = ends[g], ends[g + 1]
            Y, Z, S = R.linear_ref(X[s:e], W[g], None, "none", r[s:e])
            R.within(out[s:e], Y, R.linear_tol(Y, Z, S, 64, "none", r[s:e], out.dtype), "in place")
        # NaN and infinities of one group's rows and weights stay with it
        clean = binding.grouped_linear(X, W, offsets)
        Wn = W.clone()
        Wn[0] = float("nan")
        got = binding.grouped_linear(X, Wn, offsets)
        assert bool(got[:ends[1]].isnan().all()) and torch.equal(got[ends[1]:], clean[ends[1]:])
        Xn = X.clone()
        Xn[ends[1]] = float("inf")
        got = binding.grouped_linear(Xn, W, offsets)
        keep = torch.arange(M, device="cuda") != ends[1]
        assert torch.equal(got[keep], clean[keep]) and not bool(got[ends[1]].isfinite().any())


# --------------------------------------------------------------- backward

def check_backward(counts, N, K, dtype, kind, op_b="N", wdt=None, lead=0, tail=0, strides=False, seed=0):
    say(f"grouped backward {counts if len(counts) < 20 else len(counts)} N={N} K={K} {dtype} {kind} {op_b} dW={wdt} "
        f"lead={lead} tail={tail} strides={strides}")
    ends, offsets = offsets_of(counts, lead)
    G, M = len(counts), ends[-1] + tail
    X, dY, z = normal(seed, M, K, dtype=dtype), normal(seed + 1, M, N, dtype=dtype), normal(seed + 2, M, N, dtype=dtype)
    W = normal(seed + 3, G, K, N, dtype=dtype, scale=K ** -0.5)
    for t in (X, dY, z):
        t[ends[-1]:] = float("nan")
        t[:lead] = float("nan")
    Ws = W.transpose(1, 2).contiguous() if op_b == "T" else W
    Xs, dYs, zs = X, dY, z
    if strides:
        Xs, dYs, zs = R.padded(X, K + 3, 1)[0], R.padded(dY, N + 1, 3)[0], R.padded(z, N + 5, 1)[0]
        Ws = padded3(Ws, Ws.shape[2] + 5, 7, 3)
    pre = zs if kind != "none" else None
    dX, dW, db = binding.grouped_linear_backward(dYs, Xs, Ws, offsets, preact=pre, activation=kind,
                                                 weight_grad_dtype=wdt, op_b=op_b)
    assert dW.shape == Ws.shape and dW.dtype is (wdt or dtype)
    dX2, dW2, none = binding.grouped_linear_backward(dYs, Xs, Ws, offsets, preact=pre, activation=kind,
                                                     weight_grad_dtype=wdt, op_b=op_b, return_bias_grad=False)
    torch.cuda.synchronize()
    assert none is None and torch.equal(dW, dW2) and torch.equal(dX[lead:ends[-1]], dX2[lead:ends[-1]])
    ot = wdt or dtype
    for g, (s, e) in enumerate(zip(ends, ends[1:])):
        d = dY[s:e].double() * R.act_derivative(z[s:e].double(), kind)
        # dZ's own error: its rounding to dtype (none without an activation) and its evaluation
        ed = (R.HALF[dtype] * d.abs() + R.TINY[dtype] + 32 * R.U * dY[s:e].double().abs()) if kind != "none" else \
            torch.zeros_like(d)
        Wd, Xd = W[g].double(), X[s:e].double()
        if e > s:
            ref = d @ Wd.t()
            tol = R.HALF[dtype] * ref.abs() + R.TINY[dtype] + (ed + (N + 2) * R.U * d.abs()) @ Wd.abs().t() * 1.01
            R.within(dX[s:e], ref, tol, f"dX of group {g}")
        ref = Xd.t() @ d
        tol = R.HALF[ot] * ref.abs() + R.TINY[ot] + Xd.abs().t() @ (ed + (e - s + 2) * R.U * d.abs()) * 1.01
        R.within(dW[g].t() if op_b == "T" else dW[g], ref, tol, f"dW of group {g}")
        tol = 32 * R.U * dY[s:e].double().abs().sum(0) + (e - s + 8) * R.U * d.abs().sum(0)
        R.within(db[g], d.sum(0), tol, f"db of group {g}")


@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}g{sum(c)}r")
@pytest.mark.parametrize("op_b", ["N", "T"])
def test_backward_counts(counts, op_b):
    check_backward(counts, 136, 72, torch.bfloat16, "silu", op_b, lead=3, tail=5)
    check_backward(counts, 129, 101, torch.float16, "none", op_b, wdt=torch.float32, tail=64)


@pytest.mark.parametrize("N,K", [(1, 1), (64, 64), (7, 33), (1000, 8), (8, 1000), (257, 258), (520, 600), (66, 1002)])
@pytest.mark.parametrize("op_b", ["N", "T"])
def test_backward_sizes(N, K, op_b):
    check_backward([3, 0, 14, 1], N, K, torch.bfloat16, "gelu", op_b)
    check_backward([40, 200, 0, 90], N, K, torch.float16, "relu", op_b, wdt=torch.float32, seed=7)


@pytest.mark.parametrize("counts", [[2, 3, 1], [200, 0, 500, 131]], ids=str)
@pytest.mark.parametrize("op_b", ["N", "T"])
def test_backward_strides(counts, op_b):
    check_backward(counts, 130, 70, torch.bfloat16, "gelu", op_b, strides=True, lead=2, tail=3)
    check_backward(counts, 256, 264, torch.float16, "none", op_b, strides=True, wdt=torch.float32)


@pytest.mark.parametrize("counts,N,K", [([1500, 900, 0, 1700], 1032, 520), ([70] * 60, 512, 264), ([4100], 300, 328),
                                        ([600, 8, 1300], 2048, 2056)], ids=["4g", "many", "one", "wide"])
@pytest.mark.parametrize("op_b", ["N", "T"])
def test_backward_large(counts, N, K, op_b):
    check_backward(counts, N, K, torch.bfloat16, "gelu_tanh", op_b)
    check_backward(counts, N, K, torch.float16, "silu", op_b, wdt=torch.float32)


@pytest.mark.parametrize("kind", R.ACTS)
def test_activation_backward(kind):
    """dZ and its sums alone, with strides, in place, sums only."""
    ends, offsets = offsets_of([5, 0, 200, 64, 1], 2)
    M, N = ends[-1] + 3, 300
    for dtype in (torch.bfloat16, torch.float16):
        dY, z = normal(1, M, N, dtype=dtype), normal(2, M, N, dtype=dtype)
        pre = R.padded(z, N + 1, 3)[0] if kind != "none" else None
        out, buf = R.padded(torch.full((M, N), 7.0, dtype=dtype, device="cuda"), N + 3, 1, fill=7.0)
        dz, db = binding.grouped_activation_backward(R.padded(dY, N + 5, 1)[0], offsets, pre, kind, out=out)
        assert dz is out and bool((dz[:2] == 7.0).all()) and bool((dz[ends[-1]:] == 7.0).all())
        R.untouched(buf, M, N, N + 3, 1)
        for g, (s, e) in enumerate(zip(ends, ends[1:])):
            D = dY[s:e].double() * R.act_derivative(z[s:e].double(), kind)
            R.within(dz[s:e], D, R.HALF[dtype] * D.abs() + R.TINY[dtype] + 32 * R.U * dY[s:e].double().abs(), "dZ")
            R.within(db[g], D.sum(0), 32 * R.U * dY[s:e].double().abs().sum(0) + (e - s + 8) * R.U * D.abs().sum(0), "db")
        none, db2 = binding.grouped_activation_backward(dY, offsets, pre, kind, return_dz=False)
        assert none is None and torch.equal(db, db2)
        inplace = dY.clone()
        dz2, none = binding.grouped_activation_backward(inplace, offsets, pre, kind, out=inplace, return_bias_grad=False)
        assert dz2 is inplace and none is None
        assert torch.equal(dz2[2:ends[-1]], dz[2:ends[-1]]) and torch.equal(dz2[:2], dY[:2])


def test_gradient_against_differences():
    """grouped_linear_backward against central differences of a binary64 loss."""
    counts, N, K = [5, 0, 7], 20, 16
    ends, offsets = offsets_of(counts)
    M = ends[-1]
    X, W, dY = normal(1, M, K), normal(2, 3, K, N, scale=0.3), normal(3, M, N)
    which = torch.tensor([0] * 5 + [2] * 7, device="cuda")
    for kind in ("gelu", "gelu_tanh", "silu"):
        _, z = binding.grouped_linear(X, W, offsets, activation=kind, return_preact=True)
        dX, dW, db = binding.grouped_linear_backward(dY, X, W, offsets, preact=z, activation=kind)

        def loss(x, w, b):
            zz = torch.stack([x[i] @ w[which[i]] + b[which[i]] for i in range(M)])
            return (R.act(zz, kind) * dY.double()).sum()

        args = [X.double(), W.double(), torch.zeros(3, N, dtype=torch.float64, device="cuda")]
        h = 1e-5
        # the gradient is taken at Z rounded to bfloat16: |Z| 2^-8 |act''| of dY, and dZ's and the results' rounding
        slack = 3 * 2.0 ** -8
        zabs = (z.double().abs() * R.CURVATURE + R.LIPSCHITZ) * dY.double().abs()
        for which_arg, grad, places in ((0, dX, [(0, 0), (6, 9)]), (1, dW, [(0, 3, 4), (1, 2, 2), (2, 15, 19)]),
                                        (2, db, [(0, 1), (1, 5), (2, 13)])):
            for idx in places:
                moved = []
                for sign in (1, -1):
                    a = [t.clone() for t in args]
                    a[which_arg][idx] += sign * h
                    moved.append(loss(*a).item())
                num = (moved[0] - moved[1]) / (2 * h)
                if which_arg == 0:
                    scale = (zabs[idx[0]] @ args[1][which[idx[0]]].abs().t())[idx[1]].item()
                else:
                    rows = which == idx[0]
                    scale = (zabs[rows].sum(0)[idx[1]] if which_arg == 2 else
                             (args[0][rows].abs().t() @ zabs[rows])[idx[1:]]).item()
                assert abs(grad[idx].item() - num) <= slack * scale + 1e-6, (kind, which_arg, idx, num)


def test_streams_and_graph_replay():
    """A captured layer, forward and backward, replayed on other data and other
    offsets between eager calls gives the eager bits each time; two streams at
    once do not disturb each other."""
    for M, N, K, G in [(12, 512, 1024, 4), (200, 320, 264, 5), (2000, 640, 520, 3)]:
        say(f"grouped graph {M} {N} {K} {G}")
        X, W, b, dY = normal(1, M, K), normal(2, G, K, N, scale=K ** -0.5), normal(3, G, N), normal(4, M, N)
        gen = torch.Generator()
        gen.manual_seed(5)

        def draw():
            cuts = torch.randint(0, M + 1, (G - 1,), generator=gen).sort()[0].tolist()
            return torch.tensor([0] + cuts + [M], dtype=torch.int32).cuda()

        offsets = draw()

        def layer():
            y, z = binding.grouped_linear(X, W, offsets, bias=b, activation="gelu", return_preact=True)
            return (y, z) + tuple(binding.grouped_linear_backward(dY, X, W, offsets, preact=z, activation="gelu"))

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
            offsets.copy_(draw())
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
            outs.append(binding.grouped_linear(X, W, offsets, bias=b, activation="gelu", stream=s1))
            outs.append(binding.grouped_linear(X, W, offsets, bias=b, activation="gelu", stream=s2.cuda_stream))
        torch.cuda.synchronize()
        for o in outs:
            assert torch.equal(o, eager[0])
