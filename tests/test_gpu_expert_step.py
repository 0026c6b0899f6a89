"""A training step of a mixture's experts as a program runs it (two layers over
the rows of every expert, their backward pass, the clipping of all gradients, the
weights' gradients orthogonalised), and the experts served one by one with
weights of 4 bits: against binary64, and captured, replayed on other rows and
other offsets."""
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


class Experts:
    """Layers K -> H -> K of `groups` experts and rows for them."""

    def __init__(self, M, K, H, groups, dtype, kind):
        self.M, self.K, self.H, self.groups, self.dtype, self.kind = M, K, H, groups, dtype, kind
        self.W1 = normal(1, groups, K, H, dtype=dtype, scale=K ** -0.5)
        self.W2 = normal(2, groups, H, K, dtype=dtype, scale=H ** -0.5)
        self.b1 = normal(3, groups, H, dtype=dtype)
        self.X, self.dY = normal(4, M, K, dtype=dtype), normal(5, M, K, dtype=dtype)
        self.offsets = torch.zeros(groups + 1, dtype=torch.int32, device="cuda")
        self.gen = torch.Generator()
        self.gen.manual_seed(6)
        self.route()

    def route(self, seed=None):
        """Other rows, and other offsets with every row in a group."""
        if seed is not None:
            self.X.copy_(normal(seed, self.M, self.K, dtype=self.dtype))
            self.dY.copy_(normal(seed + 1, self.M, self.K, dtype=self.dtype))
        cuts = torch.randint(0, self.M + 1, (self.groups - 1,), generator=self.gen).sort()[0].tolist()
        self.ends = [0] + cuts + [self.M]
        self.offsets.copy_(torch.tensor(self.ends, dtype=torch.int32))

    def step(self, max_norm=1.0):
        h, z = binding.grouped_linear(self.X, self.W1, self.offsets, bias=self.b1, activation=self.kind,
                                      return_preact=True)
        y = binding.grouped_linear(h, self.W2, self.offsets, residual=self.X)
        dh, dW2, _ = binding.grouped_linear_backward(self.dY, h, self.W2, self.offsets, return_bias_grad=False)
        dX, dW1, db1 = binding.grouped_linear_backward(dh, self.X, self.W1, self.offsets, preact=z, activation=self.kind)
        before = [t.clone() for t in (dW1, dW2, db1)]
        norm = binding.clip_grad_norm([dW1, dW2, db1], max_norm)
        update = binding.newton_schulz(dW1)
        return dict(h=h, z=z, y=y, dh=dh, dX=dX, norm=norm, dW1=dW1, dW2=dW2, db1=db1, update=update), before


STEPS = [(200, 96, 160, 5, "bf16", "silu"), (37, 130, 66, 3, "f16", "gelu"), (1500, 512, 1024, 8, "bf16", "gelu_tanh"),
         (1, 64, 40, 4, "f16", "relu")]


@pytest.mark.parametrize("case", STEPS, ids=str)
def test_step(case):
    """Each result against binary64 from what its operator read."""
    M, K, H, groups, dtype, kind = *case[:4], R.DTYPES[case[4]], case[5]
    say(f"expert step {case}")
    m = Experts(M, K, H, groups, dtype, kind)
    s, before = m.step()
    torch.cuda.synchronize()
    for g, (a, e) in enumerate(zip(m.ends, m.ends[1:])):
        d = s["dh"][a:e].double() * R.act_derivative(s["z"][a:e].double(), kind)
        ed = R.HALF[dtype] * d.abs() + R.TINY[dtype] + 32 * R.U * s["dh"][a:e].double().abs()
        for x, dz, edz, got, what in ((m.X, d, ed, before[0], "dW1"),
                                      (s["h"], m.dY[a:e].double(), torch.zeros(e - a, K, device="cuda").double(),
                                       before[1], "dW2")):
            x = x[a:e].double()
            ref = x.t() @ dz
            tol = R.HALF[dtype] * ref.abs() + R.TINY[dtype] + x.abs().t() @ (edz + (e - a + 2) * R.U * dz.abs()) * 1.01
            R.within(got[g], ref, tol, f"{what} of expert {g}")
        tol = 32 * R.U * s["dh"][a:e].double().abs().sum(0) + (e - a + 8) * R.U * d.abs().sum(0)
        R.within(before[2][g], d.sum(0), tol, f"db1 of expert {g}")
        if a == e:
            continue
        Y, Z, S = R.linear_ref(m.X[a:e], m.W1[g], m.b1[g], kind, None)
        R.within(s["h"][a:e], Y, R.linear_tol(Y, Z, S, K, kind, None, dtype), f"h of expert {g}")
        R.within(s["z"][a:e], Z, R.HALF[dtype] * Z.abs() + R.TINY[dtype] + (K + 2) * R.U * S, f"z of expert {g}")
        Y, Z, S = R.linear_ref(s["h"][a:e], m.W2[g], None, "none", m.X[a:e])
        R.within(s["y"][a:e], Y, R.linear_tol(Y, Z, S, H, "none", m.X[a:e], dtype), f"y of expert {g}")
        for dz, edz, W, got, n, what in ((m.dY[a:e].double(), None, m.W2[g], s["dh"], K, "dh"),
                                         (d, ed, m.W1[g], s["dX"], H, "dX")):
            Wd = W.double()
            ref = dz @ Wd.t()
            err = (n + 2) * R.U * dz.abs() + (0 if edz is None else edz)
            R.within(got[a:e], ref, R.HALF[dtype] * ref.abs() + R.TINY[dtype] + err @ Wd.abs().t() * 1.01,
                     f"{what} of expert {g}")
    norm = math.sqrt(sum(t.double().square().sum().item() for t in before))
    assert abs(s["norm"].item() - norm) <= norm * (R.U + 1e-9)
    f = min(1.0, 1.0 / (norm + 1e-6))
    for name, b in zip(("dW1", "dW2", "db1"), before):
        ref = b.double() * f
        R.within(s[name], ref, (R.HALF[s[name].dtype] + 3.1 * R.U) * ref.abs() + R.TINY[s[name].dtype] + 2.0 ** -149, name)
    # the update of the clipped gradients, as a call of its own gives it; zeros where an expert had no row
    assert bool(s["update"].isfinite().all()) and torch.equal(s["update"], binding.newton_schulz(s["dW1"]))
    for g, (a, e) in enumerate(zip(m.ends, m.ends[1:])):
        assert a != e or not bool(s["update"][g].any())


@pytest.mark.parametrize("case", STEPS[:3], ids=str)
def test_step_replayed(case):
    M, K, H, groups, dtype, kind = *case[:4], R.DTYPES[case[4]], case[5]
    say(f"expert step replayed {case}")
    m = Experts(M, K, H, groups, dtype, kind)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m.step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured, _ = m.step()
    for seed in range(4):
        m.route(10 * seed + 20)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        kept = {k: t.clone() for k, t in captured.items()}
        eager, _ = m.step()
        torch.cuda.synchronize()
        for k, t in kept.items():
            assert torch.equal(t, eager[k]), (seed, k)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_experts_in_four_bits(dtype, kind):
    """An expert's layers with 4-bit weights, row by row, beside the grouped and
    the ordinary layer on the weights that they stand for (exact in 16 bits:
    whole multiples of a power of two): all three against one binary64."""
    dt, M, K, H, groups, size = R.DTYPES[dtype], 9, 256, 320, 3, 64
    gen = torch.Generator(device="cuda")
    gen.manual_seed(7)
    q = torch.randint(0, 16, (groups, H, K), generator=gen, device="cuda", dtype=torch.uint8)
    zeros = torch.randint(0, 16, (groups, H, K // size), generator=gen, device="cuda").to(dt)
    scales = (2.0 ** -torch.randint(5, 9, (groups, H, K // size), generator=gen, device="cuda")).to(dt)
    Q = (q[..., 0::2] | q[..., 1::2] << 4).contiguous()
    wide = lambda t: t.repeat_interleave(size, 2)
    W = wide(scales) * (q.to(dt) - wide(zeros))                       # groups x H x K
    assert torch.equal(W.double(), wide(scales).double() * (q.double() - wide(zeros).double()))
    ends = [0, 4, 4, M]
    X, b = normal(8, M, K, dtype=dt), normal(9, groups, H, dtype=dt)
    together = binding.grouped_linear(X, W, torch.tensor(ends, dtype=torch.int32, device="cuda"), bias=b, activation=kind,
                                      op_b="T")
    for g, (a, e) in enumerate(zip(ends, ends[1:])):
        if a == e:
            continue
        Y, Z, S = R.linear_ref(X[a:e], W[g].t().contiguous(), b[g], kind, None)
        tol = R.linear_tol(Y, Z, S, K, kind, None, dt)
        R.within(together[a:e], Y, tol, f"grouped, expert {g}")
        R.within(binding.linear(X[a:e], W[g], bias=b[g], activation=kind, op_b="T"), Y, tol, f"linear, expert {g}")
        # the 4-bit product adds x (16 + q) and (16 + zero) sum x
        s64 = wide(scales[g:g + 1])[0].double()
        big = s64 * (32 + q[g].double() + wide(zeros[g:g + 1])[0].double())
        S4 = X[a:e].double().abs() @ big.t().contiguous() + b[g].double().abs()
        tol4 = R.HALF[dt] * Y.abs() + R.TINY[dt] + R.LIPSCHITZ * (size + K // size + 26) * R.U * S4 + 16 * R.U * (Z.abs() + 1)
        for rows in (slice(a, a + 1), slice(a, e)):
            got = binding.linear_w4(X[rows], Q[g], scales[g], zeros=zeros[g], group_size=size, bias=b[g], activation=kind)
            n = rows.stop - rows.start
            R.within(got, Y[:n], tol4[:n], f"4 bits, expert {g}, {n} rows")
