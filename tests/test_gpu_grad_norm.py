"""The norm over many tensors and their clipping against binary64."""
from __future__ import annotations

import math

import pytest
import torch

import layer_refs as R
from gpu_support import say
from shared_memory_tiled_amd import binding

pytestmark = pytest.mark.gpu
DT = [torch.float32, torch.bfloat16, torch.float16]


def grads_of(shapes, seed=0, dtypes=DT, scale=1e-2):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return [(torch.randn(s, generator=gen, device="cuda") * scale * (1 + i % 3)).to(dtypes[i % len(dtypes)])
            for i, s in enumerate(shapes)]


def norm64(grads):
    return math.sqrt(sum(g.double().square().sum().item() for g in grads))


def check(grads, max_norm, out=None, eps=1e-6):
    """The norm within its binary32 rounding (and 1e-9 for both binary64 sums);
    values within the factor's rounding, the product's and the type's."""
    want = norm64(grads)
    before = [g.clone() for g in grads]
    norm = binding.clip_grad_norm(grads, max_norm, eps=eps, out=out)
    torch.cuda.synchronize()
    assert norm.shape == (1,) and norm.dtype is torch.float32
    assert abs(norm.item() - want) <= want * (2.0 ** -24 + 1e-9), (norm.item(), want)
    f = min(1.0, max_norm / (want + eps))
    for i, (g, b, o) in enumerate(zip(grads, before, grads if out is None else out)):
        ref = b.double() * f
        # the norm's and the factor's rounding, the product's: 3.1 units of binary32
        R.within(o, ref, R.HALF[o.dtype] * ref.abs() + R.TINY[o.dtype] + 2.0 ** -149 + 3.1 * R.U * ref.abs(), f"tensor {i}")
        if f == 1.0:
            assert torch.equal(o, b)
        if out is not None:
            assert torch.equal(g, b)
    return norm


SHAPES = [[(1,)], [()], [(4096,)], [(4097,), (0,), (4095,), (3, 5)], [(1000, 1001), (7,), (1, 1, 9)],
          [(33, 3)] * 130, [(5,)] * 300, [(2049, 1023)] * 5 + [(64,)] * 200, [(0,), (0, 4)], [(1 << 20,), (3 << 19, 3)]]


@pytest.mark.parametrize("shapes", SHAPES, ids=lambda s: f"{len(s)}x{s[0]}")
@pytest.mark.parametrize("max_norm", [0.01, 1e6, 0.0])
def test_shapes(shapes, max_norm):
    say(f"clip {len(shapes)} tensors max_norm={max_norm}")
    for dtypes in (DT, [torch.bfloat16], [torch.float32]):
        grads = grads_of(shapes, dtypes=dtypes)
        out = [torch.full_like(g, 7.0) for g in grads]
        n1 = check(grads, max_norm, out=out)
        n2 = binding.grad_norm(grads)
        kept = binding.clip_grads([g.clone() for g in grads], n2, max_norm)
        assert torch.equal(n1, n2)
        for a, b in zip(kept, out):
            assert torch.equal(a, b)
        assert torch.equal(n1, check(grads, max_norm))                 # in place
        for a, b in zip(grads, out):
            assert torch.equal(a, b)


def test_alignment_and_neighbours():
    """Tensors that begin and end anywhere in one buffer; what lies between
    them is left as it was."""
    for dtype in DT:
        buf = torch.full((200_000,), 7.0, dtype=dtype, device="cuda")
        dst = torch.full((200_001,), 7.0, dtype=dtype, device="cuda")[1:]
        mask = torch.ones_like(buf, dtype=torch.bool)
        grads, out, at = [], [], 1
        gen = torch.Generator(device="cuda")
        gen.manual_seed(3)
        for i, n in enumerate([1, 2, 7, 8, 9, 255, 4096, 4097, 8191, 12289, 20000, 3, 70001]):
            view = buf[at:at + n]
            view.copy_(torch.randn(n, generator=gen, device="cuda"))
            grads.append(view)
            out.append(dst[at:at + n])
            mask[at:at + n] = False
            at += n + 1 + i % 3
        before = [g.clone() for g in grads]
        check(grads, 0.5, out=out)
        check(grads, 0.5)
        assert bool((buf[mask] == 7.0).all()) and bool((dst[mask] == 7.0).all())
        for g, o, b in zip(grads, out, before):
            assert torch.equal(g, o) and not torch.equal(g, b)


def test_dense_layouts():
    """Transposed and permuted gradients, of their own layout."""
    base = grads_of([(300, 200), (4, 5, 6)], dtypes=[torch.bfloat16])
    grads = [base[0].t(), base[1].permute(1, 2, 0)]
    check(grads, 0.1, out=[torch.empty_like(g) for g in grads])
    check(grads, 0.1)
    with pytest.raises(ValueError):
        binding.grad_norm([base[0][:, :7]])
    with pytest.raises(ValueError):
        binding.clip_grad_norm([base[0]], 1.0, out=[torch.empty(200, 300, dtype=torch.bfloat16, device="cuda").t()])


def test_extreme_values():
    """Binary32 values whose squares pass binary32's range on either side, and
    sums that binary32 would lose."""
    for value in (1e30, 1e-30, 1e-42, 3e38):
        g = torch.full((5000,), value, device="cuda")
        want = norm64([g])
        n = binding.grad_norm([g]).item()
        if want > 3.4028235e38:
            assert n == math.inf
        else:
            assert abs(n - want) <= want * 2.0 ** -23 + 1e-45
    big = torch.ones(1 << 26, dtype=torch.bfloat16, device="cuda")
    assert binding.grad_norm([big]).item() == 8192.0
    big[1234567] = 2.0 ** 20
    want = math.sqrt((1 << 26) - 1 + 2.0 ** 40)
    assert abs(binding.grad_norm([big]).item() - want) <= want * 2.0 ** -24


def test_not_finite():
    g = torch.ones(10000, device="cuda")
    g[77] = math.inf
    n = binding.clip_grad_norm([g], 1.0)
    assert n.item() == math.inf and math.isnan(g[77].item()) and g[76].item() == 0.0
    g = torch.ones(10000, dtype=torch.float16, device="cuda")
    h = torch.ones(7, device="cuda")
    g[9999] = math.nan
    n = binding.clip_grad_norm([g, h], 1.0)
    assert math.isnan(n.item()) and bool(g.isnan().all()) and bool(h.isnan().all())


def test_listed_twice():
    g = torch.full((100,), 3.0, device="cuda")
    assert abs(binding.grad_norm([g, g]).item() - math.sqrt(1800)) < 1e-5
    with pytest.raises(binding.GemmError):
        binding.clip_grad_norm([g, g], 1.0)
    with pytest.raises(binding.GemmError):
        binding.clip_grad_norm([g, g[50:]], 1.0)
    assert bool((g == 3.0).all())
    out = [torch.empty_like(g), torch.empty_like(g)]
    binding.clip_grad_norm([g, g], 1.0, out=out)                      # read twice, written apart
    assert torch.equal(out[0], out[1])


def test_past_32_bits():
    """A tensor of more than 2^32 bytes, and more than 2^31 values."""
    n = (1 << 31) + 12345
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    for i in (0, 1 << 30, (1 << 31) - 1, 1 << 31, n - 1):
        g[i] = 3.0
    norm = binding.clip_grad_norm([g], 1.0)
    assert abs(norm.item() - math.sqrt(45)) <= 1e-5
    want = torch.tensor(3.0 / (math.sqrt(45) + 1e-6)).to(torch.bfloat16).item()
    for i in (0, 1 << 30, (1 << 31) - 1, 1 << 31, n - 1):
        assert g[i].item() == want
    assert torch.count_nonzero(g[:1 << 30]).item() == 1


def test_streams_and_graph_replay():
    """Captured clipping replayed between eager calls on other data; two
    streams at once; a norm joined from two shards."""
    grads = grads_of([(513, 129), (77,), (2000, 300)])
    out = [torch.empty_like(g) for g in grads]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        binding.clip_grad_norm(grads, 0.5, out=out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = binding.clip_grad_norm(grads, 0.5, out=out)
    for seed in range(3):
        for g, f in zip(grads, grads_of([g.shape for g in grads], seed=10 + seed)):
            g.copy_(f)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        kept = [norm.clone()] + [o.clone() for o in out]
        other = [torch.empty_like(g) for g in grads]
        eager = [binding.clip_grad_norm(grads, 0.5, out=other)] + other
        torch.cuda.synchronize()
        for a, b in zip(kept, eager):
            assert torch.equal(a, b)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    norms = [binding.grad_norm(grads, stream=s) for _ in range(4) for s in (s1, s2.cuda_stream)]
    torch.cuda.synchronize()
    for n in norms:
        assert torch.equal(n, eager[0])
    # shards: the norms of two halves joined on the GPU, then clipped by it
    a, b = binding.grad_norm(grads[:1]), binding.grad_norm(grads[1:])
    joined = torch.sqrt(a * a + b * b)
    clipped = binding.clip_grads(grads[:1], joined, 0.5, out=[torch.empty_like(grads[0])])
    want = grads[0].double() * min(1.0, 0.5 / (norm64(grads) + 1e-6))
    R.within(clipped[0], want, R.HALF[grads[0].dtype] * want.abs() + 8 * R.U * want.abs(), "shard")
