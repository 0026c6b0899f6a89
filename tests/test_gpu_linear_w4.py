"""The product with a weight held in 4 bits against binary64."""
from __future__ import annotations

import pytest
import torch

import layer_refs as R
from gpu_support import say
from shared_memory_tiled_amd import binding

pytestmark = pytest.mark.gpu


def generator(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return gen


def weight(N, K, group, dtype, zeros, seed=0, fraction=False):
    """(q N x K, packed bytes, scales, zeros): all 16 values, zero points of
    all kinds (whole numbers unless ``fraction``)."""
    gen = generator(seed)
    q = torch.randint(0, 16, (N, K), generator=gen, device="cuda", dtype=torch.uint8)
    groups = -(-K // group)
    scales = ((torch.rand(N, groups, generator=gen, device="cuda") + 0.1) * 0.1).to(dtype)
    z = None
    if zeros:
        z = torch.rand(N, groups, generator=gen, device="cuda") * 15
        z = (z if fraction else z.round()).to(dtype)
    padded = torch.nn.functional.pad(q, (0, K % 2))
    # the unused half of a last byte holds a value that must not count
    if K % 2:
        padded[:, -1] = 15
    return q, (padded[:, 0::2] | padded[:, 1::2] << 4).contiguous(), scales, z


def check(M, N, K, group, dtype, zeros=True, kind="none", bias=False, residual=False, out_dtype=None, preact=False,
          strides=False, fraction=False, seed=0, shift=0.0):
    say(f"linear_w4 M={M} N={N} K={K} group={group} {dtype} zeros={zeros} {kind} bias={bias} res={residual} "
        f"out={out_dtype} strides={strides}")
    q, Q, scales, z = weight(N, K, group, dtype, zeros, seed, fraction)
    gen = generator(seed + 1)
    X = (torch.randn(M, K, generator=gen, device="cuda") + shift).to(dtype)
    b = torch.randn(N, generator=gen, device="cuda").to(dtype) if bias else None
    ot = out_dtype or dtype
    r = torch.randn(M, N, generator=gen, device="cuda").to(ot) if residual else None
    s64 = scales.double().repeat_interleave(group, 1)[:, :K]
    z64 = z.double().repeat_interleave(group, 1)[:, :K] if zeros else torch.full_like(s64, 8.0)
    W = (s64 * (q.double() - z64)).t().contiguous()
    Y, Z, _ = R.linear_ref(X, W, b, kind, r)
    # Magnitudes that are added: x (16 + q), and (16 + z) sum x, each of which
    # the group's sum is rounded relative to; then the scaled groups, the waves
    # and the bias.
    big = (s64 * (16 + q.double())).t().contiguous() + (s64 * (16 + z64.abs())).t().contiguous()
    S = X.double().abs() @ big
    if bias:
        S = S + b.double().abs()
    terms = min(group, K) + -(-K // group) + 24
    Xs, Qs, ss, zs, rs, out, buf = X, Q, scales, z, r, None, None
    if strides:
        Xs, _ = R.padded(X, K + 3, 1)
        Qs, _ = R.padded(Q, Q.shape[1] + 5, 3, fill=255)
        ss, _ = R.padded(scales, scales.shape[1] + 1, 1)
        if zeros:
            zs, _ = R.padded(z, z.shape[1] + 2, 3)
        if residual:
            rs, _ = R.padded(r, N + 7, 1)
        out, buf = R.padded(torch.zeros(M, N, dtype=ot, device="cuda"), N + 1, 5, fill=7.0)
    got = binding.linear_w4(Xs, Qs, ss, zeros=zs, group_size=group, bias=b, activation=kind, residual=rs, out=out,
                            out_dtype=out_dtype, return_preact=preact)
    y, zz = got if preact else (got, None)
    torch.cuda.synchronize()
    err = (terms + 2) * R.U * S
    tol = R.HALF[ot] * Y.abs() + R.TINY[ot] + R.LIPSCHITZ * err
    if kind != "none":
        tol = tol + 16 * R.U * (Z.abs() + 1)
    if residual:
        tol = tol + R.U * (Y.abs() + r.double().abs())
    R.within(y, Y, tol, "out")
    if preact:
        R.within(zz, Z, R.HALF[dtype] * Z.abs() + R.TINY[dtype] + err, "preact")
    if buf is not None:
        R.untouched(buf, M, N, N + 1, 5)
    if kind == "none" and ot is torch.float32 and not residual and M * N >= 256:
        # and on average far inside it: a group of whole numbers loses bits only
        # relative to its own sums
        assert ((y.double() - Y).abs() / S.clamp(min=1e-30)).mean().item() < 3 * R.U


SIZES = [(1, 64, 64), (1, 1, 1), (1, 4096, 4096), (2, 17, 128), (3, 7, 5), (5, 33, 129), (8, 256, 2048), (15, 130, 96),
         (16, 128, 32), (17, 1000, 264), (31, 33, 4096), (32, 512, 1000), (33, 66, 40), (48, 96, 136), (63, 65, 257),
         (64, 640, 1024), (65, 70, 300), (130, 200, 515), (300, 64, 128), (1, 16, 16385), (4, 1001, 2000), (1, 8200, 130),
         (2, 16, 2047), (7, 48, 2049), (1, 5000, 127)]


@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("group", [32, 64, 128, 384, 16512])
def test_sizes(size, group):
    check(*size, group, torch.bfloat16, kind="silu", bias=True, residual=True, preact=True, seed=11)
    check(*size, group, torch.float16, zeros=False, out_dtype=torch.float32, seed=12)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_strides_and_zero_points(dtype, group):
    for M in (1, 20, 50):
        check(M, 130, 330, group, R.DTYPES[dtype], kind="gelu", bias=True, residual=True, strides=True, seed=21)
        check(M, 130, 330, group, R.DTYPES[dtype], fraction=True, strides=True, out_dtype=torch.float32, seed=22)


@pytest.mark.parametrize("kind", R.ACTS)
def test_activations(kind):
    for dtype in (torch.bfloat16, torch.float16):
        check(3, 200, 256, 64, dtype, kind=kind, bias=True, preact=True)
        check(40, 200, 256, 128, dtype, kind=kind, zeros=False)


def test_rows_far_from_zero():
    """Activations of one sign, where the sum of x is large beside the result."""
    for M in (1, 40):
        check(M, 512, 4096, 128, torch.bfloat16, shift=3.0, out_dtype=torch.float32)
        check(M, 512, 4096, 32, torch.float16, shift=3.0, zeros=False)


def test_every_value_and_place():
    """One row of X at a time picks one k: the exact weight, every value of q at
    every place of a byte, a dword and a step."""
    for dtype in (torch.bfloat16, torch.float16):
        for group in (32, 64, 128):
            N, K = 64, 256
            q, Q, scales, z = weight(N, K, group, dtype, True, seed=5)
            q[:16] = torch.arange(16, device="cuda", dtype=torch.uint8)[:, None]
            Q = (q[:, 0::2] | q[:, 1::2] << 4).contiguous()
            scales = torch.exp2(torch.randint(-3, 4, scales.shape, generator=generator(6), device="cuda").float()).to(dtype)
            want = (scales.float().repeat_interleave(group, 1) * (q.float() - z.float().repeat_interleave(group, 1)))
            eye = torch.eye(K, dtype=dtype, device="cuda")
            for rows in (1, 16, 32, 64):
                got = torch.cat([binding.linear_w4(eye[i:i + rows], Q, scales, zeros=z, group_size=group,
                                                   out_dtype=torch.float32) for i in range(0, K, rows)])
                assert torch.equal(got, want.t()), (dtype, group, rows)


def test_empty_and_no_inner():
    b = torch.randn(40, device="cuda").bfloat16()
    X = torch.zeros(5, 0, dtype=torch.bfloat16, device="cuda")
    y = binding.linear_w4(X, torch.zeros(40, 0, dtype=torch.uint8, device="cuda"),
                          torch.zeros(40, 0, dtype=torch.bfloat16, device="cuda"), bias=b, activation="silu")
    ref = R.act(b.double(), "silu").expand(5, 40)
    R.within(y, ref, R.HALF[torch.bfloat16] * ref.abs() + 1e-6, "K = 0")
    _, Q, scales, _ = weight(40, 64, 64, torch.bfloat16, False)
    X = torch.zeros(3, 64, dtype=torch.bfloat16, device="cuda")
    assert binding.linear_w4(X[:0], Q, scales, group_size=64).shape == (0, 40)
    assert binding.linear_w4(X, Q[:0], scales[:0], group_size=64).shape == (3, 0)


def test_in_place_residual_and_nan():
    q, Q, scales, z = weight(200, 256, 64, torch.float16, True)
    for M in (2, 30, 60):
        X, r = torch.randn(M, 256, device="cuda").half(), torch.randn(M, 200, device="cuda").half()
        out = r.clone()
        want = binding.linear_w4(X, Q, scales, zeros=z, group_size=64, residual=r)
        assert binding.linear_w4(X, Q, scales, zeros=z, group_size=64, residual=out, out=out) is out
        assert torch.equal(out, want)
        X[1, 70] = float("nan")                                        # stays in its row
        got = binding.linear_w4(X, Q, scales, zeros=z, group_size=64, residual=r)
        keep = torch.arange(M, device="cuda") != 1
        assert torch.equal(got[keep], want[keep]) and bool(got[1].isnan().all())
        X[1, 70] = float("inf")
        assert not bool(binding.linear_w4(X, Q, scales, zeros=z, group_size=64, residual=r)[1].isfinite().any())
    scales[7] = float("nan")                                           # and in its column
    got = binding.linear_w4(torch.ones(2, 256, device="cuda").half(), Q, scales, zeros=z, group_size=64)
    keep = torch.arange(200, device="cuda") != 7
    assert bool(got[:, 7].isnan().all()) and bool(got[:, keep].isfinite().all())


def test_refusals():
    _, Q, scales, z = weight(40, 256, 64, torch.bfloat16, True)
    X = torch.zeros(3, 256, dtype=torch.bfloat16, device="cuda")
    ok = dict(zeros=z, group_size=64)
    for bad, err in ((dict(X=X[:, :254]), ValueError), (dict(Q=Q.short()), TypeError), (dict(Q=Q[:, :100]), ValueError),
                     (dict(scales=scales.half()), TypeError), (dict(scales=scales[:, :3]), ValueError),
                     (dict(zeros=z.float()), TypeError), (dict(group_size=48), ValueError), (dict(group_size=128), ValueError),
                     (dict(X=X.float()), TypeError)):
        args = dict(X=X, Q=Q, scales=scales, **ok)
        args.update(bad)
        with pytest.raises(err):
            binding.linear_w4(**args)


def test_streams_and_graph_replay():
    q, Q, scales, z = weight(512, 1024, 128, torch.bfloat16, True)
    for M in (1, 24, 64):
        X = torch.randn(M, 1024, generator=generator(1), device="cuda").bfloat16()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            binding.linear_w4(X, Q, scales, zeros=z, activation="silu")
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            captured = binding.linear_w4(X, Q, scales, zeros=z, activation="silu")
        for seed in range(3):
            X.copy_(torch.randn(M, 1024, generator=generator(10 + seed), device="cuda"))
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            kept = captured.clone()
            eager = binding.linear_w4(X, Q, scales, zeros=z, activation="silu")
            torch.cuda.synchronize()
            assert torch.equal(kept, eager)
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        torch.cuda.synchronize()
        outs = [binding.linear_w4(X, Q, scales, zeros=z, activation="silu", stream=s) for _ in range(4)
                for s in (s1, s2.cuda_stream)]
        torch.cuda.synchronize()
        for o in outs:
            assert torch.equal(o, eager)


def test_far_apart():
    """Rows of the weight, its scales and the result whose places pass 2^32 bytes."""
    M, N, K, ld = 3, 70000, 256, 1 << 16
    say(f"linear_w4 far apart {N} {ld}")
    q, Q, scales, z = weight(N, K, 64, torch.bfloat16, True)
    X = torch.randn(M, K, generator=generator(5), device="cuda").bfloat16()
    want = binding.linear_w4(X, Q, scales, zeros=z, group_size=64)

    def far(t, ld):
        return torch.empty(t.shape[0] * ld, dtype=t.dtype, device="cuda").view(-1, ld)[:, :t.shape[1]].copy_(t)

    out = far(torch.zeros_like(want), 1 << 31)
    got = binding.linear_w4(X, far(Q, ld), far(scales, ld // 2), zeros=far(z, ld), group_size=64, out=out)
    assert got is out and torch.equal(got, want)
    W = scales.double().repeat_interleave(64, 1) * (q.double() - z.double().repeat_interleave(64, 1))
    big = scales.double().repeat_interleave(64, 1) * (32 + q.double() + z.double().repeat_interleave(64, 1))
    Y = X.double() @ W.t().contiguous()
    R.within(want, Y, R.HALF[X.dtype] * Y.abs() + 94 * R.U * (X.double().abs() @ big.t().contiguous()), "out")
