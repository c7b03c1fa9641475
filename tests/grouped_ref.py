"""The grouped operators in 64 bits, from their definitions (CPU), and their error bounds."""
from __future__ import annotations

import torch

HALF_STEP = {t: torch.finfo(t).eps / 2 for t in (torch.float32, torch.bfloat16, torch.float16)}
#: Half of the smallest step of the type: the error of a result near zero.
TINY = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


def bounds(offsets, rows):
    """Group bounds from any offsets: clamped to [0, rows], never stepping back."""
    out, top = [], 0
    for i, o in enumerate(offsets):
        o = min(max(int(o), 0), rows)
        top = o if i == 0 else max(top, o)
        out.append(top)
    return out


def gather(x, rows):
    """x[rows], a row of zeros for a number outside x."""
    if rows is None:
        return x
    rows = rows.long()
    ok = (rows >= 0) & (rows < x.shape[0])
    out = torch.zeros(rows.numel(), x.shape[1], dtype=x.dtype)
    out[ok] = x[rows[ok]]
    return out


def grouped(x, w, offsets, rows=None):
    xs = gather(x.double(), rows)
    y = torch.zeros(xs.shape[0], w.shape[2], dtype=torch.float64)
    b = bounds(offsets, xs.shape[0])
    for g in range(w.shape[0]):
        if b[g] < b[g + 1]:
            y[b[g]:b[g + 1]] = xs[b[g]:b[g + 1]] @ w[g].double()
    return y


def wgrad(x, dy, offsets, rows=None):
    xs, d = gather(x.double(), rows), dy.double()
    b = bounds(offsets, d.shape[0])
    return torch.stack([xs[b[g]:b[g + 1]].T @ d[b[g]:b[g + 1]] for g in range(len(b) - 1)])


def lora(x, w, a, b, scale, offsets, rows=None, low=None):
    """`low`: the type the product with a is rounded to."""
    xs = gather(x.double(), rows)
    y = xs @ w.double()
    e = bounds(offsets, xs.shape[0])
    for g in range(a.shape[0]):
        u = float(scale[g]) * (xs[e[g]:e[g + 1]] @ a[g].double())
        if low is not None:
            u = u.to(low).double()
        y[e[g]:e[g + 1]] += u @ b[g].double()
    out = torch.zeros_like(y)
    out[rows.long() if rows is not None else slice(None)] = y
    return out


def sum_error(dtype, terms):
    """Error of a sum of `terms` products, relative to the sum of their magnitudes.

    16-bit types: an addition of 16 products at a time, each within 2^-22 of the partial sum (the
    tensor core's additions are not rounded to nearest).  float32: the part products left out are
    below 2^-22 of a term, then eight such additions before a partial sum is taken out, and an
    addition in single precision for every 128.
    """
    if dtype == torch.float32:
        return 2.0 ** -22 + 8 * 2.0 ** -22 + (terms / 128 + 2) * 2.0 ** -24
    return (terms / 16 + 2) * 2.0 ** -22


def assert_within(got, want, magnitude, terms, extra=0.0, what=""):
    """Every entry within half a step of its type and the error of its sum; `extra`: an
    absolute error allowed on top (a tensor or a number)."""
    dtype = got.dtype
    got = got.double().cpu()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    bad_g, bad_w = ~torch.isfinite(got), ~torch.isfinite(want)
    assert torch.equal(bad_g, bad_w), f"{what}: other entries are not finite"
    sums = sum_error(dtype, terms) * magnitude + extra
    bound = HALF_STEP[dtype] * (want.abs() + sums) + sums + TINY[dtype]
    err = (got - want).abs()
    over = (err > bound) & ~bad_w
    assert not over.any(), (f"{what}: {int(over.sum())} of {over.numel()} entries beyond the bound, "
                            f"worst {float((err / bound)[~bad_w].max()):.2f} times")
