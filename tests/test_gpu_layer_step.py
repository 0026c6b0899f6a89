"""The layer operators together, as one training step of a pre-norm block
uses them: layer norm, two linear layers with their epilogues, the backward
pass through all of it, and the weights' updates orthogonalised; against the
same chain in binary64.  And places past 32 bits."""
from __future__ import annotations

import pytest
import torch

import layer_refs as R
from gpu_support import say
from shared_memory_tiled_amd import binding

pytestmark = pytest.mark.gpu


def normal(seed, *shape, dtype=torch.bfloat16, scale=1.0, shift=0.0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return (torch.randn(*shape, generator=gen, device="cuda") * scale + shift).to(dtype)


def block_step(x, g, b, W1, b1, W2, b2, dout):
    """Library: out = x + (gelu(LN(x) W1 + b1) W2 + b2), and every gradient."""
    n, mean, rstd = binding.layer_norm(x, g, b)
    h, z = binding.linear(n, W1, bias=b1, activation="gelu", return_preact=True)
    out = binding.linear(h, W2, bias=b2, residual=x)
    # second layer: its weight's gradient, and the hidden gradient through the activation
    dW2 = binding.linear(h, dout, op_a="T")
    _, db2 = binding.activation_backward(dout, return_dz=False)
    dz, db1 = binding.linear_grad(dout, W2, preact=z, activation="gelu", return_bias_grad=True)
    dn, dW1, db1_again = binding.linear_backward(dz, n, W1)
    dx, dg, db = binding.layer_norm_backward(dn, x, mean, rstd, weight=g, residual_grad=dout)
    u1, u2 = binding.newton_schulz(dW1), binding.newton_schulz(dW2)
    return dict(out=out, dW2=dW2, db2=db2, db1=db1, db1_again=db1_again, dW1=dW1, dx=dx, dg=dg, db=db, u1=u1, u2=u2)


def block_ref(x, g, b, W1, b1, W2, b2, dout):
    x, g, b, W1, b1, W2, b2, dout = (t.double() for t in (x, g, b, W1, b1, W2, b2, dout))
    n, mean, rstd, xhat = R.layer_norm_ref(x, g, b, 1e-5)
    z = n @ W1 + b1
    h = R.act(z, "gelu")
    out = h @ W2 + b2 + x
    dW2, db2 = h.t() @ dout, dout.sum(0)
    dz = (dout @ W2.t()) * R.act_derivative(z, "gelu")
    dW1, db1 = n.t() @ dz, dz.sum(0)
    dn = dz @ W1.t()
    gn = dn * g
    dx = rstd[:, None] * (gn - gn.mean(1, keepdim=True) - xhat * (gn * xhat).mean(1, keepdim=True)) + dout
    return dict(out=out, dW2=dW2, db2=db2, db1=db1, db1_again=db1, dW1=dW1, dx=dx, dg=(dn * xhat).sum(0),
                db=dn.sum(0), u1=R.newton_schulz_ref(dW1), u2=R.newton_schulz_ref(dW2))


@pytest.mark.parametrize("size", [(1, 64, 96), (40, 256, 512), (333, 200, 328), (1000, 512, 1024), (2048, 768, 1536)],
                         ids=str)
def test_training_step(size):
    """Each result passes at most eight roundings to bfloat16 on its way (LN
    out, z, h, dz, dn, ...), each of relative size HALF, and the weights'
    gradients enter the orthogonalisation, which multiplies a relative error
    of its input by at most p'(0) / p(1) ~ 5 per step in directions that are
    small in it; relative root mean squares."""
    M, D, H = size
    args = (normal(1, M, D, shift=0.3), normal(2, D, dtype=torch.float32, scale=0.1, shift=1.0),
            normal(3, D, dtype=torch.float32, scale=0.1), normal(4, D, H, scale=D ** -0.5),
            normal(5, H, scale=0.1), normal(6, H, D, scale=H ** -0.5), normal(7, D, scale=0.1), normal(8, M, D, scale=0.1))
    got, ref = block_step(*args), block_ref(*args)
    torch.cuda.synchronize()
    for name, r in ref.items():
        if name.startswith("u"):
            continue
        err = (got[name].double() - r).square().mean().sqrt() / r.square().mean().sqrt()
        say(f"{size} {name}: relative rms error {err.item():.2e}")
        assert err <= 8 * R.HALF[torch.bfloat16], (name, err)
    for name in ("u1", "u2"):                # the operator itself on the same gradient
        want = R.newton_schulz_ref(got["dW" + name[1]])
        err = (got[name].double() - want).square().mean().sqrt() / want.square().mean().sqrt()
        assert err <= R.HALF[torch.bfloat16] + 23 * 2.0 ** -12.8, (name, err)


def test_training_step_captured():
    """The step captured into a graph and replayed on changing data between
    eager steps, each replay with the eager bits."""
    M, D, H = 200, 256, 512
    args = [normal(1, M, D), normal(2, D, dtype=torch.float32, shift=1.0), normal(3, D, dtype=torch.float32),
            normal(4, D, H, scale=D ** -0.5), normal(5, H), normal(6, H, D, scale=H ** -0.5), normal(7, D), normal(8, M, D)]
    block_step(*args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = block_step(*args)
    for seed in range(3):
        args[0].copy_(normal(20 + seed, M, D))
        args[7].copy_(normal(30 + seed, M, D))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        kept = {k: v.clone() for k, v in captured.items()}
        eager = block_step(*args)
        torch.cuda.synchronize()
        for k in eager:
            assert torch.equal(kept[k], eager[k]), (seed, k)


def test_places_past_32_bits():
    """Results and inputs whose element numbers pass 2^31 and 2^32: rows far
    down agree with the same rows computed alone."""
    say("linear 70001 x 64 -> 65600")
    M, N, K = 70001, 65600, 64
    X, W, b = normal(1, M, K), normal(2, K, N, scale=K ** -0.5), normal(3, N)
    y = binding.linear(X, W, bias=b, activation="relu")
    for r0 in (0, 32760, 65530, 69990):
        Y, Z, S = R.linear_ref(X[r0:r0 + 11], W, b, "relu", None)
        R.within(y[r0:r0 + 11], Y, R.linear_tol(Y, Z, S, K, "relu", None, y.dtype), f"rows from {r0}")
    del X, W, b
    say("layer norm of the result's first 2^32 values")
    x = y[:65535, :65536]                                        # a view with a leading dimension
    rows = [0, 1, 33000, 65534]
    out, mean, rstd = binding.layer_norm(x)
    ry, rmean, rrstd, _ = R.layer_norm_ref(x[rows], None, None, 1e-5)
    R.within(out[rows], ry, R.HALF[out.dtype] * ry.abs() + 2e-3, "layer norm")
    R.within(mean[rows], rmean, 1e-5, "mean")
    dx = binding.layer_norm_backward(out, x, mean, rstd)[0]
    xhat = (x[rows].double() - mean[rows].double()[:, None]) * rstd[rows].double()[:, None]
    g = out[rows].double()
    want = rstd[rows].double()[:, None] * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    R.within(dx[rows], want, R.HALF[dx.dtype] * want.abs() + 1e-4 * rstd[rows].double()[:, None], "layer norm backward")


def test_factor_past_2_gib():
    """A weight of more than 2^31 bytes: few rows and many."""
    N, K = 33000, 34000
    W = normal(1, N, K, scale=K ** -0.5)
    for M in (3, 70):
        say(f"linear {M} x {K} -> {N}, weight stored N x K")
        X = normal(2, M, K)
        y = binding.linear(X, W, op_b="T", activation="silu")
        cols = [0, 1, 16383, 16384, 32999]
        Y, Z, S = R.linear_ref(X, W[cols].t().contiguous(), None, "silu", None)
        R.within(y[:, cols], Y, R.linear_tol(Y, Z, S, K, "silu", None, y.dtype), f"M={M}")


def test_activation_backward_rows_to_the_limit():
    """2^31 - 1 rows of one column: the last block's rows end at the type's
    last number.  Column sum over five entries that are not zero (exact)."""
    M = 2 ** 31 - 1
    say(f"activation gradient of {M} rows")
    dY = torch.zeros(M, 1, dtype=torch.bfloat16, device="cuda")
    rows = [0, 12345, 2 ** 30, M - 9, M - 1]
    for i, r in enumerate(rows):
        dY[r] = float(2 ** i)
    dz, db = binding.activation_backward(dY, activation="none")
    assert db.item() == 31.0
    assert [dz[r].item() for r in rows] == [1.0, 2.0, 4.0, 8.0, 16.0]
    assert torch.equal(dz[M - 4096:], dY[M - 4096:])


def test_column_sums_of_many_columns():
    """More columns than the column sums have blocks for at a time."""
    M, N = 3, 40_000_001
    say(f"activation gradient of {M} x {N}")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    dY = torch.randint(-8, 9, (M, N), generator=gen, device="cuda").bfloat16()
    _, db = binding.activation_backward(dY, return_dz=False)
    assert torch.equal(db, dY.float().sum(0))                    # small integers: exact
