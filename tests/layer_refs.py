"""Plain binary64 forms of the layer operators and their tolerances.

Half a rounding step relative to a value is HALF[dtype]; a binary32 sum of n
terms is within n * 2^-24 of the sum of the terms' magnitudes.
"""
from __future__ import annotations

import math

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}   # half the smallest subnormal
U = 2.0 ** -24
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
LIPSCHITZ = 1.13            # |act'| <= 1.129 (gelu near 1.41); the others are below
CURVATURE = 1.2             # |act''| <= 2 / sqrt(2 pi) + tanh form's margin, below 1.2


def act(z, kind):
    if kind == "relu":
        return torch.where(z <= 0, torch.zeros_like(z), z)
    if kind == "gelu":
        return z * torch.special.ndtr(z)
    if kind == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    if kind == "silu":
        return z * torch.sigmoid(z)
    return z


def act_derivative(z, kind):
    if kind == "relu":
        return (z > 0).to(z.dtype)
    if kind == "gelu":
        return torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        u = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        du = 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z ** 2)
        return torch.sigmoid(u) + z * torch.sigmoid(u) * torch.sigmoid(-u) * du
    if kind == "silu":
        return torch.sigmoid(z) * (1 + z * torch.sigmoid(-z))
    return torch.ones_like(z)


def within(got, ref, tol, what):
    """|got - ref| <= tol everywhere (NaN fails), with the first offender."""
    g, r = got.double(), ref.double()
    assert g.shape == r.shape, (what, g.shape, r.shape)
    bad = ~((g - r).abs() <= tol)
    if bool(bad.any()):
        i = tuple(int(x) for x in bad.nonzero()[0])
        t = tol if not isinstance(tol, torch.Tensor) else tol.expand_as(r)[i].item()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; first {i}: got {g[i].item()!r} "
                             f"ref {r[i].item()!r} tol {t!r}")


def padded(t, ld, offset=0, fill=float("nan")):
    """t's values as a view with row stride ld starting `offset` elements into
    a buffer filled with `fill`; returns (view, buffer)."""
    rows, cols = t.shape
    buf = torch.full((offset + rows * ld + 64,), fill, dtype=t.dtype, device=t.device)
    view = buf[offset:offset + rows * ld].view(rows, ld)[:, :cols]
    view.copy_(t)
    return view, buf


def untouched(buf, rows, cols, ld, offset=0, fill=7.0):
    """Everything outside the view still holds `fill`."""
    mask = torch.ones(buf.numel(), dtype=torch.bool, device=buf.device)
    mask[offset:offset + rows * ld].view(rows, ld)[:, :cols] = False
    assert bool((buf[mask] == fill).all()), "values outside the output's window were written"


# ------------------------------------------------------------------ linear

def linear_ref(X, W, bias, kind, residual):
    """(Y, Z, S): S bounds the magnitudes summed into Z."""
    Xd, Wd = X.double(), W.double()
    Z, S = Xd @ Wd, Xd.abs() @ Wd.abs()
    if bias is not None:
        Z, S = Z + bias.double(), S + bias.double().abs()
    Y = act(Z, kind)
    if residual is not None:
        Y = Y + residual.double()
    return Y, Z, S


def linear_tol(Y, Z, S, K, kind, residual, dtype):
    """Half a step of the result; the binary32 sum's error through the
    activation; the activation's own evaluation, a few operations of 2^-24
    with the exponential's argument up to |2u| <= 2 (|z| + 0.05 |z|^3): its
    error meets z e^(-2u) ..., at most 16 units of |z| + 1; a rounding of the
    residual's sum."""
    t = HALF[dtype] * Y.abs() + TINY[dtype] + LIPSCHITZ * (K + 2) * U * S
    if kind != "none":
        t = t + 16 * U * (Z.abs() + 1)
    if residual is not None:
        t = t + U * (Y.abs() + residual.double().abs())
    return t


# -------------------------------------------------------------- layer norm

def layer_norm_ref(x, w, b, eps):
    x = x.double()
    mean = x.mean(1)
    var = ((x - mean[:, None]) ** 2).mean(1)
    rstd = 1 / torch.sqrt(var + eps)
    xhat = (x - mean[:, None]) * rstd[:, None]
    y = xhat
    if w is not None:
        y = y * w.double()
    if b is not None:
        y = y + b.double()
    return y, mean, rstd, xhat


# ----------------------------------------------------------- Newton-Schulz

def newton_schulz_ref(G, steps=5, coefficients=(3.4445, -4.7750, 2.0315), eps=1e-7):
    a, b, c = coefficients
    X = G.double()
    X = X / (X.square().sum((-1, -2), keepdim=True).sqrt() + eps)
    tall = X.shape[-2] > X.shape[-1]
    for _ in range(steps):
        Xt = X.transpose(-1, -2).contiguous()
        S = Xt @ X if tall else X @ Xt
        P = b * S + c * (S @ S)
        X = a * X + (X @ P if tall else P @ X)
    return X
