"""Routing to experts and log probabilities in 64 bits, from their definitions (CPU), and their error
bounds."""
from __future__ import annotations

import math

import torch

from grouped_ref import HALF_STEP, TINY

STEP = 2.0 ** -24        # half a step of FP32, relative


def scores(logits, score):
    """softmax or sigmoid of every row; -inf gives 0, and a row of nothing else zeros."""
    x = logits.double()
    if score == "sigmoid":
        return torch.sigmoid(x)
    m = x.amax(1, keepdim=True)
    e = torch.where(x == -math.inf, 0.0, torch.exp(x - torch.where(m == -math.inf, 0.0, m)))
    s = e.sum(1, keepdim=True)
    return torch.where(s == 0, 0.0, e / s)


def log_scores(logits, score):
    x = logits.double()
    if score == "sigmoid":
        return torch.nn.functional.logsigmoid(x)
    return x - torch.logsumexp(x, 1, keepdim=True)


def route(logits, k, bias=None, score="softmax", groups=1, top_groups=1, group_best=1,
          renormalise=True, scale=1.0):
    """(experts, weights) of rows without NaN."""
    x = logits.double()
    T, E = x.shape
    s = scores(logits, score)
    c = s if bias is None else s + bias.double()
    order = x if bias is None else c
    shut = x == -math.inf
    if bias is not None:
        shut |= (bias == -math.inf)[None]
    experts = torch.full((T, k), -1, dtype=torch.int32)
    weights = torch.zeros(T, k, dtype=torch.float64)
    size = E // groups
    for t in range(T):
        live = [e for e in range(E) if not shut[t, e]]
        if top_groups < groups:
            worth = {}
            for e in live:
                worth.setdefault(e // size, []).append(
                    float(c[t, e]) if bias is not None or group_best == 2 else float(x[t, e]))
            value = {g: sum(sorted(v, reverse=True)[:group_best]) for g, v in worth.items()}
            best = sorted(value, key=lambda g: (-value[g], g))[:top_groups]
            live = [e for e in live if e // size in best]
        live.sort(key=lambda e: (-float(order[t, e]), e))
        mine = live[:k]
        if not mine:
            continue
        experts[t, :len(mine)] = torch.tensor(mine, dtype=torch.int32)
        if renormalise:
            weights[t, :len(mine)] = scale * torch.softmax(log_scores(logits[t:t + 1], score)[0, mine],
                                                           0)
        else:
            weights[t, :len(mine)] = scale * s[t, mine]
    return experts, weights


def weight_bound(logits, experts, weights):
    """Absolute error of the weights: an exponential's argument is rounded (by at most half a step
    of the distance from the row's maximum) and its value within two steps, a sum has at most 32 + 5
    additions, and a quotient and a product are rounded: (|t| + 48) half steps of the weight."""
    x = logits.double()
    reach = (x.amax(1, keepdim=True) - x).clamp(max=120).nan_to_num(0.0, 0.0, 0.0)
    mine = reach.gather(1, experts.long().clamp(min=0))
    return weights.abs() * (mine + 48) * STEP + 2.0 ** -140


def route_grad(dweights, logits, experts, score="softmax", renormalise=True, scale=1.0):
    """(dlogits, sums of the magnitudes of the terms) from the formulas."""
    s = scores(logits, score)
    T, E = s.shape
    d, size = torch.zeros(T, E, dtype=torch.float64), torch.zeros(T, E, dtype=torch.float64)
    for t in range(T):
        at = [(j, int(e)) for j, e in enumerate(experts[t]) if 0 <= e < E]
        if not at:
            continue
        e = torch.tensor([a[1] for a in at])
        g = scale * dweights[t, [a[0] for a in at]].double()
        if renormalise:
            lg = log_scores(logits[t:t + 1], score)[0, e]
            w = torch.softmax(lg, 0) if bool((lg > -math.inf).any()) else torch.zeros(len(at)).double()
            v = w * (g - (g * w).sum())
            big = w * (g.abs() + (g * w).abs().sum())
            if score == "sigmoid":
                v, big = v * (1 - s[t, e]), big * (1 - s[t, e])
            d[t].index_add_(0, e, v)
            size[t].index_add_(0, e, big)
        elif score == "sigmoid":
            v = g * s[t, e] * (1 - s[t, e])
            d[t].index_add_(0, e, v)
            size[t].index_add_(0, e, g.abs() * s[t, e])
        else:
            ds = torch.zeros(E, dtype=torch.float64).index_add_(0, e, g)
            dot = (g * s[t, e]).sum()
            d[t] = s[t] * (ds - dot)
            size[t] = s[t] * (torch.zeros(E, dtype=torch.float64).index_add_(0, e, g.abs())
                              + (g * s[t, e]).abs().sum())
    return d, size


def logprobs(logits, tokens=None, top=0, scale=1.0):
    """A dict of the outputs, and of the means of |t| and t^2 that the bounds need; rows without NaN
    and +inf."""
    x = logits.double() * scale
    T, V = x.shape
    out = {"lse": torch.full((T,), -math.inf, dtype=torch.float64),
           "entropy": torch.zeros(T, dtype=torch.float64),
           "logprob": torch.zeros(T, dtype=torch.float64),
           "top_ids": torch.full((T, top), -1, dtype=torch.int32),
           "top_logprobs": torch.full((T, top), -math.inf, dtype=torch.float64)}
    mean, square, log_s = (torch.zeros(T, dtype=torch.float64) for _ in range(3))
    for r in range(T):
        live = x[r] > -math.inf
        if bool(live.any()):
            m = x[r].max()
            t = (x[r] - m)[live]
            s = torch.exp(t).sum()
            p = torch.exp(t) / s
            log_s[r] = torch.log(s)
            out["lse"][r] = m + log_s[r]
            out["entropy"][r] = log_s[r] - (p * t.clamp(min=-2000)).sum()
            mean[r], square[r] = (p * t.abs()).sum(), (p * t * t).nan_to_num(0.0).sum()
        lp = (x[r] - m) - log_s[r] if bool(live.any()) else torch.full((V,), -math.inf).double()
        if tokens is not None and 0 <= int(tokens[r]) < V:
            out["logprob"][r] = lp[int(tokens[r])]
        if top:
            order = torch.argsort(logits[r].double(), descending=True, stable=True)
            order = [int(i) for i in order if bool(live[i])][:top]
            out["top_ids"][r, :len(order)] = torch.tensor(order, dtype=torch.int32)
            out["top_logprobs"][r, :len(order)] = lp[order]
    return out, mean, square, log_s


def logprob_bounds(out, mean, square, log_s, cols):
    """Absolute errors of (lse, logprob-like values, entropy).

    A term e^t: its argument is two roundings off (of the difference and of the product with c, whose
    own rounding is a third), 3 |t| half steps, and the exponential is within 2^-22.  Sums: a thread
    of a block adds at most cols / 512 + 32 terms (16 a round of 4 vectors, 8192 columns a round), one
    of the warp that does a row alone, of up to 8192 columns, cols / 64 + 32 (1024 columns a round); and
    40 more join threads, warps and blocks.
    """
    depth = (cols / 64 if cols <= 8192 + 15 else cols / 512) + 72
    s_err = depth * STEP + 3 * mean * STEP + 2.0 ** -22
    w_err = mean * (depth * STEP + 2.0 ** -22) + 4 * square * STEP
    log_err = s_err + 2 * STEP * (1 + log_s.abs())
    lse = log_err + 2 * STEP * out["lse"].abs().nan_to_num(0.0, 0.0, 0.0)
    ent = log_err + w_err + mean * s_err + 4 * STEP * (1 + mean + out["entropy"])
    return lse, log_err, ent


def logprob_grad(logits, tokens, lse, dlogprob=None, entropy=None, dentropy=None, top_ids=None,
                 dtop=None, scale=1.0):
    """(dlogits, bounds before the result's rounding)."""
    x = logits.double() * scale
    T, V = x.shape
    zero = torch.zeros(T, 1, dtype=torch.float64)
    lse = lse.double()[:, None]
    dead = lse == -math.inf
    lp = torch.where(dead, -math.inf, x - torch.where(dead, 0.0, lse))
    p = torch.exp(lp)
    low = lp.clamp(min=-2000)
    hot, size = torch.zeros(T, V, dtype=torch.float64), torch.zeros(T, V, dtype=torch.float64)
    total = zero.clone()
    if dlogprob is not None:
        given = (tokens >= 0) & (tokens < V)
        g = torch.where(given, dlogprob.double(), 0.0)[:, None]
        hot.scatter_add_(1, torch.where(given, tokens, 0).long()[:, None], g)
        total = total + g
        size = size + g.abs()
    if dtop is not None:
        given = (top_ids >= 0) & (top_ids < V)
        e = torch.where(given, dtop.double(), 0.0)
        hot.scatter_add_(1, torch.where(given, top_ids, 0).long(), e)
        total = total + e.sum(1, keepdim=True)
        size = size + e.abs().sum(1, keepdim=True)
    h = dentropy.double()[:, None] if dentropy is not None else zero
    ent = entropy.double()[:, None] if dentropy is not None else zero
    d = hot - p * (total + h * (low + ent))
    # p: the exponent's two roundings and the exponential; the sum of up to 33 gradients.
    err = p * ((4 * low.abs() + 8) * STEP * (size + h.abs() * (low.abs() + ent.abs()))
               + 33 * STEP * size)
    err = err + 40 * STEP * hot.abs()
    quiet = dead | ((total == 0) & (h == 0))
    d = torch.where(dead, 0.0, torch.where(quiet, hot, d)) * scale
    return d, (err * scale).clamp(min=0)


def assert_close(got, want, error, what=""):
    """Within the error and the rounding to the result's type; not finite in the same places."""
    step = HALF_STEP[got.dtype]
    g = got.double().cpu()
    assert g.shape == want.shape, (what, g.shape, want.shape)
    odd = ~torch.isfinite(want)
    assert torch.equal(g[odd].nan_to_num(7e300), want[odd].nan_to_num(7e300)), what
    bound = (step * (want.abs() + error) + error + TINY[got.dtype])[~odd]
    off = (g - want).abs()[~odd]
    assert not bool((off > bound).any()), (
        f"{what}: {int((off > bound).sum())} of {off.numel()} beyond the bound, worst "
        f"{float((off / bound).max()):.2f} times")
