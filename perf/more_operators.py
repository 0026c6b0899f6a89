"""Cases that measure the fully connected layer's further forms: the layer whose
rows belong to experts with a weight each, with its backward pass; the global
norm of a model's gradients and their clipping; the product of a few rows with
a weight held in 4 bits.

``listed()`` names the cases, ``draw()`` makes more of the same ranges,
``prepare()`` puts a case's inputs on the GPU, ``run()`` makes one pass: the
plain form in elementary torch operations (``own`` false) or the library's
entry points (``own`` true).  ``exact()`` computes the same outputs in
binary64 from the definitions.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
CLIP_EPS = 1e-6


def listed():
    return [
        # eight tokens of a decoder, two experts of sixteen each: the chosen
        # experts' weights are read once and that read is the time
        dict(name="grouped_linear_16x2048x4096_e16_bf16", op="grouped_linear", groups=16, M=16, N=2048, K=4096,
             dtype="bf16", trans_b=True, bias=False, activation="silu", preact=False),
        # a short prompt over many small experts, some of them without a row
        dict(name="grouped_linear_4096x1024x2048_e64_bf16", op="grouped_linear", groups=64, M=4096, N=1024, K=2048,
             dtype="bf16", trans_b=False, bias=False, activation="silu", preact=False),
        # a small ragged layer, trained: biases, pre-activation kept
        dict(name="grouped_linear_999x2002x1000_e7_f16", op="grouped_linear", groups=7, M=999, N=2002, K=1000,
             dtype="f16", trans_b=False, bias=True, activation="gelu", preact=True),
        # a training batch, two experts of eight per token
        dict(name="grouped_linear_16384x4096x4096_e8_bf16", op="grouped_linear", groups=8, M=16384, N=4096, K=4096,
             dtype="bf16", trans_b=False, bias=False, activation="gelu_tanh", preact=True),
        # the backward pass of a small ragged layer
        dict(name="grouped_linear_backward_1000x500x2000_e6_f16", op="grouped_linear_backward", groups=6, M=1000,
             N=500, K=2000, dtype="f16", trans_b=True, activation="silu", bias=True),
        # the backward pass of a training batch, sixteen experts
        dict(name="grouped_linear_backward_8192x2048x4096_e16_bf16", op="grouped_linear_backward", groups=16, M=8192,
             N=2048, K=4096, dtype="bf16", trans_b=False, activation="gelu_tanh", bias=False),
        # a small model's gradients, all binary32: latency and launches
        dict(name="clip_grad_norm_4x64_f32", op="clip_grad_norm", layers=4, width=64, hidden=200, vocab=500,
             dtype="f32", max_norm=0.25),
        # an ordinary model: bfloat16 matrices beside binary32 vectors
        dict(name="clip_grad_norm_12x896_bf16", op="clip_grad_norm", layers=12, width=896, hidden=3584, vocab=16001,
             dtype="bf16", max_norm=1.0),
        # a large one: 0.8 billion values
        dict(name="clip_grad_norm_16x2048_bf16", op="clip_grad_norm", layers=16, width=2048, hidden=8192, vocab=8000,
             dtype="bf16", max_norm=1.0),
        # one token against a square projection held in 4 bits
        dict(name="linear_w4_1x4096x4096_bf16", op="linear_w4", M=1, N=4096, K=4096, group_size=128, dtype="bf16",
             zeros=False, bias=False, activation="none", residual=False),
        # ragged sizes: an odd number of outputs, a last group that is half full
        dict(name="linear_w4_3x1001x2000_bf16", op="linear_w4", M=3, N=1001, K=2000, group_size=32, dtype="bf16",
             zeros=True, bias=True, activation="silu", residual=False),
        # a decoding batch against a wide projection, onto the residual stream
        dict(name="linear_w4_16x8192x8192_f16", op="linear_w4", M=16, N=8192, K=8192, group_size=64, dtype="f16",
             zeros=True, bias=False, activation="none", residual=True),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["grouped_linear", "grouped_linear", "grouped_linear_backward", "clip_grad_norm", "linear_w4"])
    if op in ("grouped_linear", "grouped_linear_backward"):
        while True:
            groups = _log_int(rng, 1, 64)
            M = _log_int(rng, 1 if op == "grouped_linear" else 64, 16384)
            N, K = _log_int(rng, 64, 8192), _log_int(rng, 64, 8192)
            if rng.random() < 0.6:                     # most layers' widths are multiples of 8
                N, K = -(-N // 8) * 8, -(-K // 8) * 8
            if M * N * K <= 8192 * 2048 * 4096 * (2 if op == "grouped_linear" else 1) and groups * N * K <= 1 << 27:
                break
        case = dict(op=op, groups=groups, M=M, N=N, K=K, dtype=rng.choice(["bf16", "f16"]),
                    trans_b=rng.random() < 0.5, activation=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]),
                    bias=rng.random() < 0.5)
        if op == "grouped_linear":
            case["preact"] = rng.random() < 0.5
        return case
    if op == "clip_grad_norm":
        while True:
            case = dict(op=op, layers=_log_int(rng, 1, 32), width=_log_int(rng, 32, 2048),
                        hidden=_log_int(rng, 64, 8192), vocab=_log_int(rng, 100, 32000),
                        dtype=rng.choice(["bf16", "f16", "f32"]), max_norm=rng.choice([0.1, 1.0, 1.0, 100.0]))
            if sum(math.prod(shape) for shape, _ in _grad_shapes(case)) * (2 if case["dtype"] == "f32" else 1) < 8e8:
                return case
    while True:
        M, N, K = _log_int(rng, 1, 64), _log_int(rng, 64, 16384), _log_int(rng, 64, 16384)
        if rng.random() < 0.6:
            N, K = -(-N // 64) * 64, -(-K // 64) * 64
        if N * K <= 8192 * 8192:
            return dict(op=op, M=M, N=N, K=K, group_size=rng.choice([32, 64, 128]), dtype=rng.choice(["bf16", "f16"]),
                        zeros=rng.random() < 0.5, bias=rng.random() < 0.5,
                        activation=rng.choice(["none", "none", "gelu_tanh", "silu"]), residual=rng.random() < 0.5)


def _grad_shapes(case):
    """(shape, dtype name) of a model's gradients: matrices of the case's
    type, vectors in binary32."""
    D, H, t = case["width"], case["hidden"], case["dtype"]
    shapes = [((case["vocab"], D), t)]
    for _ in range(case["layers"]):
        shapes += [((D,), "f32"), ((D,), "f32"), ((D, D), t), ((D, 2 * D), t), ((D,), "f32"), ((D, D), t),
                   ((D, H), t), ((H,), "f32"), ((H, D), t), ((D,), "f32")]
    return shapes


def _flat_sizes(case):
    """Values of each type among a model's gradients."""
    sizes = {}
    for shape, t in _grad_shapes(case):
        sizes[t] = sizes.get(t, 0) + math.prod(shape)
    return sizes


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, shift=0.0, to=dtype):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale + shift).to(to)

    s = dict(case=case)
    op = case["op"]
    if op in ("grouped_linear", "grouped_linear_backward"):
        G, M, N, K = case["groups"], case["M"], case["N"], case["K"]
        # rows sorted by expert; some experts are several times as popular as others
        host = torch.Generator()
        host.manual_seed(seed)
        popularity = torch.softmax(0.7 * torch.randn(G, generator=host), 0)
        chosen = torch.multinomial(popularity, M, replacement=True, generator=host)
        ends = torch.cumsum(torch.bincount(chosen, minlength=G), 0)
        s["bounds"] = [0] + ends.tolist()              # the plain form's copy on the host
        s["offsets"] = torch.tensor(s["bounds"], dtype=torch.int32, device="cuda")
        s["X"] = normal(M, K)
        s["W"] = normal(G, *((N, K) if case["trans_b"] else (K, N)), scale=K ** -0.5)
        if op == "grouped_linear":
            s["bias"] = normal(G, N, scale=0.5) if case["bias"] else None
        else:
            s["dY"] = normal(M, N, scale=0.1)
            s["preact"] = normal(M, N) if case["activation"] != "none" else None
    elif op == "clip_grad_norm":
        # each tensor at a scale of its own
        s["grads"] = [normal(*shape, scale=1e-3 * math.exp(0.5 * math.sin(7.0 * i + seed)), to=DTYPES[t])
                      for i, (shape, t) in enumerate(_grad_shapes(case))]
        # the clipped ones in one buffer per type, as a sharded optimiser keeps them
        s["flat"] = {t: torch.empty(n, dtype=DTYPES[t], device="cuda") for t, n in _flat_sizes(case).items()}
        s["clipped"], at = [], dict.fromkeys(s["flat"], 0)
        for shape, t in _grad_shapes(case):
            n = math.prod(shape)
            s["clipped"].append(s["flat"][t][at[t]:at[t] + n].view(shape))
            at[t] += n
    else:
        M, N, K, size = case["M"], case["N"], case["K"], case["group_size"]
        s["X"] = normal(M, K)
        W = normal(N, K, scale=K ** -0.5, to=torch.float32)
        blocks = -(-K // size)
        Wg = torch.nn.functional.pad(W, (0, blocks * size - K)).view(N, blocks, size)
        if case["zeros"]:                              # from the group's range
            low, high = Wg.amin(2).clamp(max=0), Wg.amax(2).clamp(min=0)
            s["scales"] = ((high - low) / 15).clamp(min=1e-6).to(dtype)
            s["zeros"] = torch.round(-low / s["scales"].float()).clamp(0, 15).to(dtype)
            zero = s["zeros"].float()[:, :, None]
        else:                                          # symmetric about 8
            s["scales"] = (Wg.abs().amax(2) / 7).clamp(min=1e-6).to(dtype)
            s["zeros"] = None
            zero = 8.0
        q = torch.round(Wg / s["scales"].float()[:, :, None] + zero).clamp(0, 15).to(torch.uint8)
        q = torch.nn.functional.pad(q.view(N, -1)[:, :K], (0, K % 2))
        s["Q"] = (q[:, 0::2] | (q[:, 1::2] << 4)).contiguous()       # the even k in the low half of a byte
        s["bias"] = normal(N, scale=0.5) if case["bias"] else None
        s["residual"] = normal(M, N) if case["residual"] else None
    return s


# ------------------------------------------------------------ plain form

def _activate(z, kind):
    if kind == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if kind == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if kind == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if kind == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _activate_derivative(z, kind):
    if kind == "relu":
        return (z > 0).to(z.dtype)
    if kind == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if kind == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)
    if kind == "silu":
        sig = 1.0 / (1.0 + torch.exp(-z))
        return sig * (1.0 + z * (1.0 - sig))
    return torch.ones_like(z)


def _plain(s):
    case = s["case"]
    op, dtype = case["op"], DTYPES[case["dtype"]]
    if op == "grouped_linear":
        z = torch.empty(case["M"], case["N"], dtype=torch.float32, device="cuda")
        for g, (b, e) in enumerate(zip(s["bounds"], s["bounds"][1:])):
            if e > b:
                W = s["W"][g].float()
                z[b:e] = s["X"][b:e].float() @ (W.t() if case["trans_b"] else W)
                if s["bias"] is not None:
                    z[b:e] += s["bias"][g].float()
        y = _activate(z, case["activation"]).to(dtype)
        return (y, z.to(dtype)) if case["preact"] else (y,)
    if op == "grouped_linear_backward":
        dz = s["dY"].float()
        if s["preact"] is not None:
            dz = dz * _activate_derivative(s["preact"].float(), case["activation"])
        dX = torch.empty(case["M"], case["K"], dtype=torch.float32, device="cuda")
        dW = torch.zeros(s["W"].shape, dtype=torch.float32, device="cuda")
        db = torch.zeros(case["groups"], case["N"], dtype=torch.float32, device="cuda")
        for g, (b, e) in enumerate(zip(s["bounds"], s["bounds"][1:])):
            if e > b:
                W, X, d = s["W"][g].float(), s["X"][b:e].float(), dz[b:e]
                dX[b:e] = d @ (W if case["trans_b"] else W.t())
                dW[g] = d.t() @ X if case["trans_b"] else X.t() @ d
                db[g] = d.sum(0)
        return (dX.to(dtype), dW.to(dtype)) + ((db,) if case["bias"] else ())
    if op == "clip_grad_norm":
        # the squares' sum in 64 bits: many values
        total = torch.zeros((), dtype=torch.float64, device="cuda")
        for g in s["grads"]:
            total = total + (g.float() * g.float()).sum(dtype=torch.float64)
        norm = total.sqrt()
        factor = (case["max_norm"] / (norm + CLIP_EPS)).clamp(max=1.0).float()
        for g, out in zip(s["grads"], s["clipped"]):
            out.copy_((g.float() * factor).to(g.dtype))
        return norm.float().reshape(1), *s["flat"].values()
    K, size = case["K"], case["group_size"]
    q = torch.stack((s["Q"] & 15, s["Q"] >> 4), 2).view(case["N"], -1)[:, :K].float()
    scale = s["scales"].float().repeat_interleave(size, 1)[:, :K]
    zero = 8.0 if s["zeros"] is None else s["zeros"].float().repeat_interleave(size, 1)[:, :K]
    z = s["X"].float() @ (scale * (q - zero)).t()
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _activate(z, case["activation"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return (y.to(dtype),)


# ------------------------------------------------------------ the library

def _library(s):
    from shared_memory_tiled_amd import binding
    case = s["case"]
    op = case["op"]
    if op == "grouped_linear":
        out = binding.grouped_linear(s["X"], s["W"], s["offsets"], bias=s["bias"], activation=case["activation"],
                                     return_preact=case["preact"], op_b="T" if case["trans_b"] else "N")
        return tuple(out) if case["preact"] else (out,)
    if op == "grouped_linear_backward":
        out = binding.grouped_linear_backward(s["dY"], s["X"], s["W"], s["offsets"], preact=s["preact"],
                                              activation=case["activation"], op_b="T" if case["trans_b"] else "N",
                                              return_bias_grad=case["bias"])
        return tuple(out) if case["bias"] else tuple(out[:2])
    if op == "clip_grad_norm":
        norm = binding.clip_grad_norm(s["grads"], case["max_norm"], eps=CLIP_EPS, out=s["clipped"])
        return norm, *s["flat"].values()
    return (binding.linear_w4(s["X"], s["Q"], s["scales"], zeros=s["zeros"], group_size=case["group_size"],
                              bias=s["bias"], activation=case["activation"], residual=s["residual"]),)


def run(state):
    return _library(state) if own else _plain(state)


# ------------------------------------------------------------ work, exact

def work(case):
    op = case["op"]
    e = 4 if case["dtype"] == "f32" else 2
    if op in ("grouped_linear", "grouped_linear_backward"):
        G, M, N, K = case["groups"], case["M"], case["N"], case["K"]
        # weights of experts that some row chose; their number for equal popularity
        used = G * (1.0 - (1.0 - 1.0 / G) ** M)
        if op == "grouped_linear":
            return {"bytes": int(e * (M * K + used * K * N + M * N * (1 + case["preact"]) + used * N * case["bias"])),
                    "flops": 2 * M * N * K}
        ins = M * N * (1 + (case["activation"] != "none")) + M * K + used * K * N
        return {"bytes": int(e * (ins + M * K + G * K * N) + 4 * G * N * case["bias"]), "flops": 4 * M * N * K}
    if op == "clip_grad_norm":
        values = [(math.prod(shape), 4 if t == "f32" else 2) for shape, t in _grad_shapes(case)]
        return {"bytes": sum(2 * n * size for n, size in values) + 4, "flops": sum(3 * n for n, _ in values)}
    M, N, K = case["M"], case["N"], case["K"]
    blocks = -(-K // case["group_size"])
    return {"bytes": N * -(-K // 2) + e * (M * K + M * N * (1 + case["residual"]) + N * case["bias"]
                                           + N * blocks * (1 + case["zeros"])),
            "flops": 2 * M * N * K}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "clip_grad_norm":
        norm = torch.linalg.vector_norm(torch.stack([torch.linalg.vector_norm(g.double()) for g in s["grads"]]))
        factor = min(1.0, case["max_norm"] / (norm.item() + CLIP_EPS))
        flat = {t: [] for t in s["flat"]}
        for g, (_, t) in zip(s["grads"], _grad_shapes(case)):
            flat[t].append(g.double().mul_(factor).view(-1))
        return norm.reshape(1), *[torch.cat(parts) for parts in flat.values()]
    kind = case["activation"]

    def phi(z):                                          # normal distribution function
        return torch.special.ndtr(z)

    def activated(z):
        if kind == "relu":
            return z.clamp(min=0)
        if kind == "gelu":
            return z * phi(z)
        if kind == "gelu_tanh":                          # 1 + tanh(u) = 2 / (1 + exp(-2 u))
            return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
        if kind == "silu":
            return z * torch.sigmoid(z)
        return z

    if op == "linear_w4":
        N, K, size = case["N"], case["K"], case["group_size"]
        q = torch.zeros(N, 2 * s["Q"].shape[1], dtype=torch.float64, device="cuda")
        q[:, 1::2] = (s["Q"].int() // 16).double()
        q[:, 0::2] = (s["Q"].int() % 16).double()
        z = torch.zeros(case["M"], N, dtype=torch.float64, device="cuda")
        for i in range(s["scales"].shape[1]):            # group by group
            part = slice(i * size, min(K, (i + 1) * size))
            centred = q[:, part] - (8.0 if s["zeros"] is None else s["zeros"][:, i:i + 1].double())
            z += torch.mm(s["X"][:, part].double(), (centred * s["scales"][:, i:i + 1].double()).t().contiguous())
        if s["bias"] is not None:
            z += s["bias"].double()
        y = activated(z)
        return (y if s["residual"] is None else y + s["residual"].double(),)
    G, M, N, K = case["groups"], case["M"], case["N"], case["K"]
    expert = torch.bucketize(torch.arange(M, device="cuda"), s["offsets"][1:].long(), right=True)   # of each row
    if op == "grouped_linear":
        z = torch.empty(M, N, dtype=torch.float64, device="cuda")
        for g in range(G):
            rows = (expert == g).nonzero()[:, 0]
            W = s["W"][g].double()
            z[rows] = torch.mm(s["X"][rows].double(), W.t().contiguous() if case["trans_b"] else W)
        if s["bias"] is not None:
            z += s["bias"].double()[expert]
        return (activated(z), z) if case["preact"] else (activated(z),)
    dz = s["dY"].double()
    if s["preact"] is not None:
        z = s["preact"].double()
        if kind == "relu":
            dz = torch.where(z > 0, dz, torch.zeros_like(dz))
        elif kind == "gelu":
            dz = dz * (phi(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
        elif kind == "gelu_tanh":
            u = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
            sg = torch.sigmoid(u)
            dz = dz * (sg + z * sg * torch.sigmoid(-u) * 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * z ** 2))
        elif kind == "silu":
            sg = torch.sigmoid(z)
            dz = dz * (sg + z * sg * torch.sigmoid(-z))
    dX = torch.empty(M, K, dtype=torch.float64, device="cuda")
    dW = torch.empty(s["W"].shape, dtype=torch.float64, device="cuda")
    for g in range(G):
        rows = (expert == g).nonzero()[:, 0]
        W, X, d = s["W"][g].double(), s["X"][rows].double(), dz[rows]
        dX[rows] = torch.mm(d, W if case["trans_b"] else W.t().contiguous())
        dW[g] = torch.mm(d.t().contiguous(), X) if case["trans_b"] else torch.mm(X.t().contiguous(), d)
    if not case["bias"]:
        return dX, dW
    return dX, dW, torch.zeros(G, N, dtype=torch.float64, device="cuda").index_add_(0, expert, dz)
