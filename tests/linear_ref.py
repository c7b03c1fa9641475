"""Linear layers in 64 bits, from their definitions (CPU), and their error bounds."""
from __future__ import annotations

import math

import torch

import grouped_ref
from grouped_ref import HALF_STEP, TINY, sum_error

ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
ROOT = math.sqrt(2 / math.pi)


def act(z, kind):
    if kind == "relu":
        return torch.where(z < 0, 0.0, z)
    if kind == "silu":
        return z * torch.sigmoid(z)
    if kind == "gelu":
        return 0.5 * z * torch.erfc(-z * math.sqrt(0.5))
    if kind == "gelu_tanh":
        return z * torch.sigmoid(2 * ROOT * (z + 0.044715 * z ** 3))
    return z


def slope(z, kind):
    if kind == "relu":
        return (z > 0).to(z.dtype)
    if kind == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * torch.sigmoid(-z))
    if kind == "gelu":
        return 0.5 * torch.erfc(-z * math.sqrt(0.5)) + z * torch.exp(-z * z / 2) / math.sqrt(
            2 * math.pi)
    if kind == "gelu_tanh":
        u = 2 * ROOT * (z + 0.044715 * z ** 3)
        s = torch.sigmoid(u)
        return s * (1 + z * torch.sigmoid(-u) * 2 * ROOT * (1 + 3 * 0.044715 * z * z))
    return torch.ones_like(z)


def act_error(z, y):
    """Of an activation's evaluation, absolute.  Its exponent or erfc argument is off by a few roundings
    of an argument that grows as z^2 (gelu's) or |z| (silu's), or z^4 (the tanh form's cubic times z,
    whose value there is 0 or z but for e^-|u|, u |z| at least: bounded by its maximum); the hardware's
    exponential and quotient add a few 2^-22."""
    z = z.abs().clamp(max=13.0)
    return y.abs() * (3 * z * z + 2 * z + 12) * 2.0 ** -22 + 2.0 ** -100


def forward(x, w, bias, kind, residual):
    """(y, z, error of y, error of z) before rounding to the result's type."""
    dtype, K = x.dtype, x.shape[1]
    xd, wd = x.double(), w.double()
    z = xd @ wd
    err = sum_error(dtype, max(K, 1)) * (xd.abs() @ wd.abs())
    if bias is not None:
        z = z + bias.double()
        err = err + 2.0 ** -24 * z.abs()
    y = act(z, kind)
    y_err = 1.2 * err + act_error(z, y) if kind not in ("none", "relu") else err
    if residual is not None:
        y = y + residual.double()
        y_err = y_err + 2.0 ** -24 * y.abs()
    return y, z, y_err, err


def assert_close(got, want, error, what=""):
    dtype = got.dtype
    g = got.double().cpu()
    assert g.shape == want.shape, (what, g.shape, want.shape)
    odd = ~torch.isfinite(want)
    assert torch.equal(~torch.isfinite(g), odd), f"{what}: other entries are not finite"
    bound = (HALF_STEP[dtype] * (want.abs() + error) + error + TINY[dtype])[~odd]
    off = (g - want).abs()[~odd]
    assert not bool((off > bound).any()), (
        f"{what}: {int((off > bound).sum())} of {off.numel()} beyond the bound, worst "
        f"{float((off / bound).max()):.2f} times")


def backward(dy, x, w, z, kind):
    """({dx, dw, dbias}, their errors before rounding): dz is rounded to the type for the products."""
    dtype = dy.dtype
    d = dy.double()
    dz, dz_err = d, torch.zeros_like(d)
    if kind != "none":
        zd = z.double()
        dz = d * slope(zd, kind)
        if kind != "relu":
            near = zd.abs().clamp(max=13.0)
            dz_err = d.abs() * (1 + near) * (3 * near * near + 2 * near + 12) * 2.0 ** -22
    rounded = dz_err + (HALF_STEP[dtype] * dz.abs() + TINY[dtype] if kind != "none" else 0.0)
    xd, wd = x.double(), w.double()
    M, N = dy.shape
    out = {"dx": dz @ wd.T, "dw": xd.T @ dz, "dbias": dz.sum(0)}
    size = dz.abs() + rounded
    err = {"dx": sum_error(dtype, max(N, 1)) * (size @ wd.abs().T) + rounded @ wd.abs().T,
           "dw": sum_error(dtype, max(M, 1)) * (xd.abs().T @ size) + xd.abs().T @ rounded,
           "dbias": dz_err.sum(0) + (M / 8 + 80) * 2.0 ** -24 * dz.abs().sum(0)}
    return out, err


__all__ = ["ACTS", "act", "slope", "forward", "backward", "assert_close", "grouped_ref"]
