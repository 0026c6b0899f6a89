"""Cases that measure the operators of a fully connected layer's training and
serving path: the product with bias, activation and residual in its epilogue,
its backward pass, layer norm with its backward pass, and the Newton-Schulz
orthogonalisation of a weight's update.

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
EPS = 1e-5                                   # layer norm
NS_COEFFICIENTS = (3.4445, -4.7750, 2.0315)  # quintic with a steep start, not a fixed point at 1
NS_EPS = 1e-7


def listed():
    return [
        # one token of a decoder against a square projection: the weight is
        # read once and latency decides
        dict(name="linear_1x4096x4096_bf16", op="linear", M=1, N=4096, K=4096, dtype="bf16", trans_b=False,
             bias=True, activation="silu", residual=False, preact=False),
        # a decoding batch: output projection onto the residual stream, weight stored N x K
        dict(name="linear_24x8192x4096_f16", op="linear", M=24, N=8192, K=4096, dtype="f16", trans_b=True,
             bias=True, activation="none", residual=True, preact=False),
        # a short prompt in ragged sizes, trained: pre-activation kept
        dict(name="linear_999x2002x1000_bf16", op="linear", M=999, N=2002, K=1000, dtype="bf16", trans_b=False,
             bias=True, activation="gelu", residual=False, preact=True),
        # a training batch's hidden layer
        dict(name="linear_8192x4096x4096_bf16", op="linear", M=8192, N=4096, K=4096, dtype="bf16", trans_b=False,
             bias=True, activation="gelu_tanh", residual=False, preact=True),
        # the backward pass of a small ragged layer
        dict(name="linear_backward_1000x500x2000_f16", op="linear_backward", M=1000, N=500, K=2000, dtype="f16",
             trans_b=False, activation="silu"),
        # the backward pass of a training batch's hidden layer
        dict(name="linear_backward_8192x4096x4096_bf16", op="linear_backward", M=8192, N=4096, K=4096, dtype="bf16",
             trans_b=False, activation="gelu_tanh"),
        # a few tokens of a decoder
        dict(name="layer_norm_8x4096_bf16", op="layer_norm", M=8, N=4096, dtype="bf16", affine=True),
        # a training batch with wide rows
        dict(name="layer_norm_8192x8192_bf16", op="layer_norm", M=8192, N=8192, dtype="bf16", affine=True),
        # binary32 rows of ragged width
        dict(name="layer_norm_backward_1000x1001_f32", op="layer_norm_backward", M=1000, N=1001, dtype="f32",
             affine=True, residual=False),
        # a training batch, with the gradient that comes past the layer
        dict(name="layer_norm_backward_8192x4096_bf16", op="layer_norm_backward", M=8192, N=4096, dtype="bf16",
             affine=True, residual=True),
        # four tall weights of one shape, binary32 momentum
        dict(name="newton_schulz_4x2000x1000_f32", op="newton_schulz", batch=4, M=2000, N=1000, dtype="f32", steps=5),
        # one square weight, bfloat16 momentum
        dict(name="newton_schulz_4096x4096_bf16", op="newton_schulz", batch=1, M=4096, N=4096, dtype="bf16", steps=5),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_backward", "layer_norm", "layer_norm_backward", "newton_schulz"])
    if op in ("linear", "linear_backward"):
        while True:
            M = _log_int(rng, 1 if op == "linear" else 64, 8192)
            N, K = _log_int(rng, 64, 8192), _log_int(rng, 64, 8192)
            if rng.random() < 0.6:                     # most layers' widths are multiples of 8
                N, K = -(-N // 8) * 8, -(-K // 8) * 8
            if M * N * K <= 8192 * 4096 * 4096:
                break
        case = dict(op=op, M=M, N=N, K=K, dtype=rng.choice(["bf16", "f16"]), trans_b=rng.random() < 0.5,
                    activation=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]))
        if op == "linear":
            case.update(bias=rng.random() < 0.7, residual=rng.random() < 0.5, preact=rng.random() < 0.5)
        return case
    if op in ("layer_norm", "layer_norm_backward"):
        while True:
            M, N = _log_int(rng, 1 if op == "layer_norm" else 16, 16384), _log_int(rng, 32, 16384)
            dtype = rng.choice(["bf16", "f16", "f32"])
            if M * N * (2 if dtype == "f32" else 1) <= 8192 * 4096:
                break
        case = dict(op=op, M=M, N=N, dtype=dtype, affine=rng.random() < 0.8)
        if op == "layer_norm_backward":
            case["residual"] = rng.random() < 0.5
        return case
    while True:
        batch = rng.choice([1, 1, 2, 3, 4, 8])
        M, N = _log_int(rng, 16, 4096), _log_int(rng, 16, 4096)
        if batch * M * N * min(M, N) <= 1 << 33:
            return dict(op=op, batch=batch, M=M, N=N, dtype=rng.choice(["bf16", "f16", "f32"]), steps=5)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, shift=0.0, to=dtype):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale + shift).to(to)

    s = dict(case=case)
    op, M, N = case["op"], case["M"], case["N"]
    if op in ("linear", "linear_backward"):
        K = case["K"]
        s["X"] = normal(M, K)
        s["W"] = normal(*((N, K) if case["trans_b"] else (K, N)), scale=K ** -0.5)
        if op == "linear":
            s["bias"] = normal(N, scale=0.5) if case["bias"] else None
            s["residual"] = normal(M, N) if case["residual"] else None
        else:
            s["dY"] = normal(M, N, scale=0.1)
            s["preact"] = normal(M, N) if case["activation"] != "none" else None
    elif op in ("layer_norm", "layer_norm_backward"):
        s["X"] = normal(M, N, scale=2.0, shift=0.5)
        s["weight"] = normal(N, scale=0.2, shift=1.0, to=torch.float32) if case["affine"] else None
        s["bias"] = normal(N, scale=0.2, to=torch.float32) if case["affine"] else None
        if op == "layer_norm_backward":
            s["dY"] = normal(M, N, scale=0.1)
            s["residual_grad"] = normal(M, N, scale=0.1) if case["residual"] else None
            x = s["X"].double()
            s["mean"] = x.mean(1).float()
            s["rstd"] = (x.var(1, unbiased=False) + EPS).rsqrt().float()
    else:                                   # momentum: a few strong directions over a broad rest
        B = case["batch"]
        strong = torch.randn(B, M, 8, generator=gen, device="cuda") @ torch.randn(B, 8, N, generator=gen, device="cuda")
        rest = torch.randn(B, M, N, generator=gen, device="cuda")
        s["G"] = (1e-3 * (0.1 * strong + rest)).to(dtype)
        if B == 1:
            s["G"] = s["G"][0]
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
    if op == "linear":
        W = s["W"].float()
        z = s["X"].float() @ (W.t() if case["trans_b"] else W)
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _activate(z, case["activation"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return (y.to(dtype), z.to(dtype)) if case["preact"] else (y.to(dtype),)
    if op == "linear_backward":
        X, W, dz = s["X"].float(), s["W"].float(), s["dY"].float()
        if s["preact"] is not None:
            dz = dz * _activate_derivative(s["preact"].float(), case["activation"])
        if case["trans_b"]:
            dX, dW = dz @ W, dz.t() @ X
        else:
            dX, dW = dz @ W.t(), X.t() @ dz
        return dX.to(dtype), dW.to(dtype), dz.sum(0)
    if op == "layer_norm":
        x = s["X"].float()
        mean = x.sum(1, keepdim=True) / case["N"]
        centred = x - mean
        rstd = torch.rsqrt((centred * centred).sum(1, keepdim=True) / case["N"] + EPS)
        y = centred * rstd
        if s["weight"] is not None:
            y = y * s["weight"] + s["bias"]
        return y.to(dtype), mean[:, 0], rstd[:, 0]
    if op == "layer_norm_backward":
        dy, rstd = s["dY"].float(), s["rstd"][:, None]
        xhat = (s["X"].float() - s["mean"][:, None]) * rstd
        g = dy * s["weight"] if s["weight"] is not None else dy
        n = case["N"]
        dx = rstd * (g - g.sum(1, keepdim=True) / n - xhat * ((g * xhat).sum(1, keepdim=True) / n))
        if s["residual_grad"] is not None:
            dx = dx + s["residual_grad"].float()
        if s["weight"] is None:
            return (dx.to(dtype),)
        return dx.to(dtype), (dy * xhat).sum(0), dy.sum(0)
    X = s["G"].float()
    wide = case["M"] <= case["N"]
    if not wide:
        X = X.transpose(-1, -2).contiguous()
    # the norm in 64 bits: a sum of many squares of small values
    norm = s["G"].double().square().sum((-1, -2), keepdim=True).sqrt()
    X = X * (1.0 / (norm + NS_EPS)).float()
    a, b, c = NS_COEFFICIENTS
    for _ in range(case["steps"]):
        A = X @ X.transpose(-1, -2).contiguous()
        B = b * A + c * (A @ A)
        X = a * X + B @ X
    if not wide:
        X = X.transpose(-1, -2).contiguous()
    return (X.to(dtype),)


# ------------------------------------------------------------ the library

def _library(s):
    from shared_memory_tiled_amd import binding
    case = s["case"]
    op = case["op"]
    if op == "linear":
        out = binding.linear(s["X"], s["W"], bias=s["bias"], activation=case["activation"], residual=s["residual"],
                             return_preact=case["preact"], op_b="T" if case["trans_b"] else "N")
        return tuple(out) if case["preact"] else (out,)
    if op == "linear_backward":
        return tuple(binding.linear_backward(s["dY"], s["X"], s["W"], preact=s["preact"],
                                             activation=case["activation"], op_b="T" if case["trans_b"] else "N"))
    if op == "layer_norm":
        return tuple(binding.layer_norm(s["X"], s["weight"], s["bias"], eps=EPS))
    if op == "layer_norm_backward":
        out = binding.layer_norm_backward(s["dY"], s["X"], s["mean"], s["rstd"], weight=s["weight"],
                                          residual_grad=s["residual_grad"])
        return tuple(out) if case["affine"] else (out[0],)
    return (binding.newton_schulz(s["G"], steps=case["steps"], coefficients=NS_COEFFICIENTS, eps=NS_EPS),)


def run(state):
    return _library(state) if own else _plain(state)


# ------------------------------------------------------------ work, exact

def work(case):
    op, M, N = case["op"], case["M"], case["N"]
    e = 4 if case["dtype"] == "f32" else 2
    if op == "linear":
        K = case["K"]
        outs = 1 + case["preact"] + case["residual"]
        return {"bytes": e * (M * K + K * N + outs * M * N + case["bias"] * N), "flops": 2 * M * N * K}
    if op == "linear_backward":
        K = case["K"]
        ins = M * N * (1 + (case["activation"] != "none")) + M * K + K * N
        return {"bytes": e * (ins + M * K + K * N) + 4 * N, "flops": 4 * M * N * K}
    if op == "layer_norm":
        return {"bytes": 2 * e * M * N + 8 * M + 8 * N * case["affine"], "flops": 8 * M * N}
    if op == "layer_norm_backward":
        planes = 3 + case["residual"]
        return {"bytes": planes * e * M * N + 8 * M + 12 * N * case["affine"], "flops": 12 * M * N}
    m, n = min(M, N), max(M, N)
    # two of the three products of a step are symmetric: half their entries
    return {"bytes": 2 * e * case["batch"] * M * N,
            "flops": case["batch"] * case["steps"] * (3 * m * m * n + m * m * m)}


def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    op = case["op"]
    if op in ("linear", "linear_backward"):
        W = d["W"].t().contiguous() if case["trans_b"] else d["W"]          # K x N

        def phi(z):                                                          # normal distribution function
            return torch.special.ndtr(z)

        kind = case["activation"]
        if op == "linear":
            z = torch.mm(d["X"], W)
            if d["bias"] is not None:
                z += d["bias"]
            if kind == "relu":
                y = z.clamp(min=0)
            elif kind == "gelu":
                y = z * phi(z)
            elif kind == "gelu_tanh":        # 1 + tanh(u) = 2 / (1 + exp(-2 u))
                y = z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
            elif kind == "silu":
                y = z * torch.sigmoid(z)
            else:
                y = z
            if d["residual"] is not None:
                y = y + d["residual"]
            return (y, z) if case["preact"] else (y,)
        dz = d["dY"]
        if d["preact"] is not None:
            z = d["preact"]
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
        dW = torch.mm(d["X"].t().contiguous(), dz)
        return torch.mm(dz, W.t().contiguous()), dW.t().contiguous() if case["trans_b"] else dW, dz.sum(0)
    if op == "layer_norm":
        var, mean = torch.var_mean(d["X"], 1, unbiased=False)
        rstd = 1 / torch.sqrt(var + EPS)
        y = (d["X"] - mean[:, None]) * rstd[:, None]
        if d["weight"] is not None:
            y = torch.addcmul(d["bias"], y, d["weight"])
        return y, mean, rstd
    if op == "layer_norm_backward":
        # the gradient with the given statistics: (g - <g> - xhat <g xhat>) / sigma
        xhat = torch.sub(d["X"], d["mean"][:, None]).mul_(d["rstd"][:, None])
        g = d["dY"] if d["weight"] is None else d["dY"] * d["weight"]
        dx = g - g.mean(1, keepdim=True)
        dx -= xhat * (g * xhat).mean(1, keepdim=True)
        dx *= d["rstd"][:, None]
        if d["residual_grad"] is not None:
            dx += d["residual_grad"]
        if d["weight"] is None:
            return (dx,)
        return dx, torch.sum(d["dY"] * xhat, 0), d["dY"].sum(0)
    G = d["G"] if case["batch"] > 1 else d["G"][None]
    a, b, c = NS_COEFFICIENTS
    out = torch.empty_like(G)
    for i in range(G.shape[0]):                       # X <- X (a I + b S + c S^2), S the smaller Gram matrix
        X = G[i] / (torch.linalg.matrix_norm(G[i]) + NS_EPS)
        tall = X.shape[0] > X.shape[1]
        for _ in range(case["steps"]):
            Xt = X.t().contiguous()
            S = torch.mm(Xt, X) if tall else torch.mm(X, Xt)
            P = torch.mm(S, c * S).add_(S, alpha=b)
            P.diagonal().add_(a)
            X = torch.mm(X, P) if tall else torch.mm(P, X)
        out[i] = X
    return (out if case["batch"] > 1 else out[0],)
