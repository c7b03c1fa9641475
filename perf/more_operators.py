"""Measured cases of the operators around a model's products: routing to experts, a product with bias,
activation and residual, log probabilities of given tokens, and the gradients of all three.

Each case is a dict of plain values with an ``op``:

* ``route``: experts and weights of every token from its scores (softmax or sigmoid of the logits),
  chosen with a bias for balance and within the best groups of experts;
* ``route_grad``: the gradient of the weights with respect to the logits;
* ``gemm_bias_act``: y = act(x w + bias) + residual, with w (K, N) or (``trans``) stored (N, K), and,
  for training, z = x w + bias beside it;
* ``gemm_bias_act_grad``: the gradients with respect to x, w and bias from dy and z;
* ``logprob``: every row's log probability of its given token, entropy, log of the sum of
  exponentials, and its ``top`` most probable tokens;
* ``logprob_grad``: the gradient with respect to the logits.

``run`` computes them in plain torch operations in 32 bits, or through this package where ``own``
is true.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}


def listed():
    return [
        # One decode step of 5 requests through a small mixture: latency only.
        {"name": "route 5 tokens 8 experts", "op": "route", "tokens": 5, "experts": 8, "k": 2,
         "groups": 1, "top_groups": 1, "group_best": 1, "score": "softmax", "bias": False,
         "dtype": "fp32"},
        # A training batch over many experts, chosen within groups and balanced by a bias.
        {"name": "route 16384 tokens 256 experts", "op": "route", "tokens": 16384, "experts": 256,
         "k": 8, "groups": 8, "top_groups": 4, "group_best": 2, "score": "sigmoid", "bias": True,
         "dtype": "fp32"},
        # The backward pass of an odd number of tokens.
        {"name": "route grad 1001 tokens 60 experts", "op": "route_grad", "tokens": 1001,
         "experts": 60, "k": 4, "score": "softmax", "renormalise": False, "dtype": "bf16"},
        # The backward pass of the training batch.
        {"name": "route grad 16384 tokens 256 experts", "op": "route_grad", "tokens": 16384,
         "experts": 256, "k": 8, "score": "sigmoid", "renormalise": True, "dtype": "fp32"},
        # One token through a projection: reading the weights is all there is.
        {"name": "linear 1 token bf16", "op": "gemm_bias_act", "tokens": 1, "K": 4096, "N": 4096,
         "act": "silu", "bias": True, "residual": True, "pre": False, "trans": True,
         "dtype": "bf16"},
        # A training batch: the forward pass of a layer, its z kept for the backward pass.
        {"name": "linear 8192 tokens bf16", "op": "gemm_bias_act", "tokens": 8192, "K": 4096,
         "N": 4096, "act": "gelu", "bias": True, "residual": True, "pre": True, "trans": False,
         "dtype": "bf16"},
        # Its backward pass, a smaller batch.
        {"name": "linear grad 4096 tokens bf16", "op": "gemm_bias_act_grad", "tokens": 4096,
         "K": 4096, "N": 4096, "act": "gelu", "bias": True, "trans": False, "dtype": "bf16"},
        # Single precision at odd sizes.
        {"name": "linear grad 1001 rows fp32", "op": "gemm_bias_act_grad", "tokens": 1001,
         "K": 1000, "N": 2047, "act": "silu", "bias": True, "trans": True, "dtype": "fp32"},
        # A decode batch: the chosen tokens' log probabilities, and the alternatives to show.
        {"name": "logprob 32 rows 131072 tokens", "op": "logprob", "tokens": 32, "vocab": 131072,
         "top": 20, "dtype": "bf16", "padded": False},
        # Scoring a batch of whole texts under a large vocabulary.
        {"name": "logprob 4096 rows 131072 tokens", "op": "logprob", "tokens": 4096,
         "vocab": 131072, "top": 0, "dtype": "bf16", "padded": True},
        # Single precision, an odd vocabulary, gradients of log probability and entropy.
        {"name": "logprob grad 515 rows 50001 tokens", "op": "logprob_grad", "tokens": 515,
         "vocab": 50001, "dtype": "fp32", "entropy": True, "padded": True},
        # The backward pass of a training batch, log probabilities alone.
        {"name": "logprob grad 4096 rows 65536 tokens", "op": "logprob_grad", "tokens": 4096,
         "vocab": 65536, "dtype": "bf16", "entropy": False, "padded": True},
    ]


def _between(rng, lo, hi):
    """A size between lo and hi, its logarithm spread evenly; odd ones among them."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A matrix dimension: three in four 1, 1.25 or 1.75 times a power of two, the others odd."""
    v = _between(rng, lo, hi)
    if rng.random() < 0.25:
        return v | 1
    steps = [int(m * 2 ** e) for e in range(6, 18) for m in (1, 1.25, 1.75)]
    return min((s for s in steps if lo <= s <= hi), key=lambda s: abs(math.log(s / v)))


def _cost(case):
    """A case's work in seconds, roughly: what its bytes or its operations take."""
    w = work(case)
    rate = 2e14 if case["dtype"] == "fp32" else 1.5e15
    if case["op"] == "logprob":
        return w["bytes"] / 6e12 * (1 + case["top"] / 16)     # the plain form's share of `top`
    if not case["op"].startswith("gemm"):
        return w["bytes"] / 6e12
    return max(w["bytes"] / 6e12, w["flops"] / rate)


def draw(rng):
    op = rng.choice(["route", "route_grad", "gemm_bias_act", "gemm_bias_act",
                     "gemm_bias_act_grad", "logprob", "logprob", "logprob_grad"])
    most = max(_cost(c) for c in listed() if c["op"].split("_")[0] == op.split("_")[0])
    while True:
        case = {"op": op, "dtype": rng.choice(["bf16", "fp16", "fp32"])}
        if op.startswith("route"):
            case["tokens"] = _between(rng, 1, 16384)
            case["score"] = rng.choice(["softmax", "sigmoid"])
            case["experts"] = rng.choice([8, 16, 60, 64, 128, 160, 256, 384, 512])
            case["k"] = rng.choice([1, 2, 4, 6, 8])
            if op == "route_grad":
                case["renormalise"] = rng.random() < 0.5
            else:
                case["groups"] = rng.choice([1, 1, 2, 4, 8])
                if case["experts"] % case["groups"]:
                    continue
                case["top_groups"] = rng.randint(1, case["groups"])
                case["group_best"] = rng.choice([1, 2])
                case["bias"] = rng.random() < 0.5
                if case["k"] > case["experts"] // case["groups"] * case["top_groups"]:
                    continue
        elif op.startswith("gemm"):
            case["tokens"] = _between(rng, 1, 8192)
            case["K"], case["N"] = _width(rng, 64, 8192), _width(rng, 64, 8192)
            case["act"] = rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"])
            case["bias"] = rng.random() < 0.6
            case["trans"] = rng.random() < 0.5
            if op == "gemm_bias_act":
                case["residual"] = rng.random() < 0.5
                case["pre"] = rng.random() < 0.3
        else:
            case["tokens"] = _between(rng, 1, 8192)
            case["vocab"] = _width(rng, 1000, 163840)
            case["padded"] = rng.random() < 0.5
            if op == "logprob":
                case["top"] = rng.choice([0, 0, 1, 5, 20])
            else:
                case["entropy"] = rng.random() < 0.5
        if _cost(case) <= most:
            return case


def work(case):
    op, t, size = case["op"], case["tokens"], _BYTES[case["dtype"]]
    if op == "route":
        e, k = case["experts"], case["k"]
        return {"bytes": float(t * e * size + 8 * t * k + (4 * e if case["bias"] else 0)),
                "flops": 8.0 * t * e}
    if op == "route_grad":
        e, k = case["experts"], case["k"]
        # (The sigmoid's gradient, and the softmax's where the weights are made to add up to one,
        # need the chosen logits alone.)
        read = e if case["score"] == "softmax" and not case["renormalise"] else k
        return {"bytes": float(t * (e + read) * size + 8 * t * k), "flops": 4.0 * t * (read + k)}
    if op.startswith("gemm"):
        K, N = case["K"], case["N"]
        x, w, y = t * K, K * N, t * N
        bias = 4.0 * N if case["bias"] else 0.0
        if op == "gemm_bias_act":
            return {"bytes": size * float(x + w + y * (1 + case["residual"] + case["pre"])) + bias,
                    "flops": 2.0 * t * K * N}
        return {"bytes": size * float(2 * x + 2 * w + y * (1 + (case["act"] != "none"))) + bias,
                "flops": 4.0 * t * K * N}
    v = case["vocab"]
    if op == "logprob":
        return {"bytes": float(t * v * size + t * (4 + 12 + 8 * case["top"])),
                "flops": 6.0 * t * v}
    return {"bytes": float(2 * t * v * size + t * (16 + 4 * case["entropy"])), "flops": 6.0 * t * v}


# ---- inputs --------------------------------------------------------------------------------


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, dtype, t = case["op"], _TYPES[case["dtype"]], case["tokens"]
    state = dict(case)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, device="cuda", generator=gen) * std).to(dtype)

    if op.startswith("route"):
        e, k = case["experts"], case["k"]
        popular = 0.5 * torch.randn(e, device="cuda", generator=gen)
        logits = 1.2 * torch.randn(t, e, device="cuda", generator=gen) + popular
        state["logits"] = logits.to(dtype)
        if op == "route":
            # A bias for balance: against an expert's popularity, in steps of a training run.
            state["bias"] = None
            if case["bias"]:
                state["bias"] = (-0.1 * popular / 0.001).round() * 0.001
        else:
            state["chosen"] = state["logits"].float().topk(k, dim=1).indices.to(torch.int32)
            state["dweights"] = torch.randn(t, k, device="cuda", generator=gen) * 0.1
        return state
    if op.startswith("gemm"):
        K, N = case["K"], case["N"]
        state["x"] = normal(t, K)
        state["w"] = normal(N, K, std=K ** -0.5).t() if case["trans"] else normal(
            K, N, std=K ** -0.5)
        if op == "gemm_bias_act":
            state["bias"] = None
            if case["bias"]:
                state["bias"] = torch.randn(N, device="cuda", generator=gen) * 0.2
            state["residual"] = normal(t, N) if case["residual"] else None
        else:
            state["dy"] = normal(t, N)
            state["z"] = None if case["act"] == "none" else normal(t, N)
        return state
    v = case["vocab"]
    logits = normal(t, v, std=2.5)
    # The tokens are probable ones, as those that a model chose or learns; some rows are padding.
    tokens = torch.randint(0, v, (t,), device="cuda", generator=gen)
    logits[torch.arange(t, device="cuda"), tokens] += 8.0
    if case["padded"] and t > 1:
        tokens[torch.rand(t, device="cuda", generator=gen) < 0.1] = -1
    state["logits"], state["tokens"] = logits, tokens
    if op == "logprob_grad":
        m = logits.amax(1, keepdim=True).float()
        p = torch.exp(logits.float() - m)
        s = p.sum(1, keepdim=True)
        state["lse"] = (m + s.log())[:, 0]
        state["entropy_of"] = (s.log() - (p * (logits.float() - m)).sum(1, keepdim=True) / s)[:, 0]
        state["dlogprob"] = torch.randn(t, device="cuda", generator=gen)
        state["dentropy"] = (0.01 * torch.randn(t, device="cuda", generator=gen)
                             if case["entropy"] else None)
    return state


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(state):
    import tiled_matrix_multiply_gb300 as tmm
    op = state["op"]
    if op == "route":
        r = tmm.route_rows(state["logits"], state["k"], bias=state["bias"], score=state["score"],
                           groups=state["groups"], top_groups=state["top_groups"],
                           group_best=state["group_best"], scale=2.5)
        return {"experts": r.experts, "weights": r.weights}
    if op == "route_grad":
        return tmm.route_rows_grad(state["dweights"], state["logits"], state["chosen"],
                                   score=state["score"], renormalise=state["renormalise"],
                                   scale=2.5)
    if op == "gemm_bias_act":
        return tmm.gemm_bias_act(state["x"], state["w"], bias=state["bias"], act=state["act"],
                                 residual=state["residual"], pre=state["pre"])
    if op == "gemm_bias_act_grad":
        g = tmm.gemm_bias_act_grad(state["dy"], state["x"], state["w"], pre=state["z"],
                                   act=state["act"], dbias=state["bias"])
        return {"dx": g.dx, "dw": g.dw, "dbias": g.dbias} if state["bias"] else {"dx": g.dx,
                                                                                 "dw": g.dw}
    if op == "logprob":
        r = tmm.logprob_rows(state["logits"], state["tokens"], top=state["top"])
        out = {"logprob": r.logprob, "entropy": r.entropy, "lse": r.lse}
        if state["top"]:
            out.update(top_ids=r.top_ids, top_logprobs=r.top_logprobs)
        return out
    return tmm.logprob_rows_grad(state["logits"], state["tokens"], state["lse"],
                                 dlogprob=state["dlogprob"], entropy=state["entropy_of"],
                                 dentropy=state["dentropy"])


# ---- the plain forms ---------------------------------------------------------------------


def _run_plain(state):
    op = state["op"]
    if op == "route":
        return _plain_route(state["logits"], state["bias"], state["k"], state["groups"],
                            state["top_groups"], state["group_best"], state["score"], 2.5)
    if op == "route_grad":
        return _plain_route_grad(state["dweights"], state["logits"], state["chosen"].long(),
                                 state["score"], state["renormalise"], 2.5)
    if op == "gemm_bias_act":
        z = state["x"].float() @ state["w"].float()
        if state["bias"] is not None:
            z = z + state["bias"]
        y = _plain_act(z, state["act"])
        if state["residual"] is not None:
            y = y + state["residual"].float()
        dtype = state["x"].dtype
        return (y.to(dtype), z.to(dtype)) if state["pre"] else y.to(dtype)
    if op == "gemm_bias_act_grad":
        dtype = state["x"].dtype
        dz = state["dy"].float()
        if state["act"] != "none":
            dz = dz * _plain_slope(state["z"].float(), state["act"])
        out = {"dx": (dz @ state["w"].float().t()).to(dtype),
               "dw": (state["x"].float().t() @ dz).to(dtype)}
        if state["bias"]:
            out["dbias"] = dz.sum(0)
        return out
    if op == "logprob":
        return _plain_logprob(state["logits"], state["tokens"], state["top"])
    return _plain_logprob_grad(state["logits"], state["tokens"], state["lse"],
                               state["entropy_of"], state["dlogprob"], state["dentropy"])


def _plain_scores(x, score):
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    p = torch.exp(x - x.amax(1, keepdim=True))
    return p / p.sum(1, keepdim=True)


def _plain_route(logits, bias, k, groups, top_groups, group_best, score, scale):
    t, e = logits.shape
    # The choice in 64 bits: two experts' scores may be closer than 32 bits tell apart.
    c = _plain_scores(logits.double(), score)
    if bias is not None:
        c = c + bias.double()
    value = c if bias is not None else logits.double()
    if top_groups < groups:
        best = torch.sort(c.view(t, groups, -1), dim=2, descending=True).values
        order = torch.sort(best[..., :group_best].sum(2), dim=1, descending=True,
                           stable=True).indices
        open_ = torch.zeros(t, groups, dtype=torch.bool, device=c.device)
        open_.scatter_(1, order[:, :top_groups], True)
        value = torch.where(open_.repeat_interleave(e // groups, dim=1), value, -math.inf)
    chosen = torch.sort(value, dim=1, descending=True, stable=True).indices[:, :k]
    w = _plain_scores(logits.float(), score).gather(1, chosen)
    w = w / w.sum(1, keepdim=True) * scale
    return {"experts": chosen.to(torch.int32), "weights": w}


def _plain_route_grad(dweights, logits, chosen, score, renormalise, scale):
    s = _plain_scores(logits.float(), score)
    g = dweights * scale
    if renormalise:
        mine = s.gather(1, chosen)
        total = mine.sum(1, keepdim=True)
        g = (g - (g * mine).sum(1, keepdim=True) / total) / total
    ds = torch.zeros_like(s).scatter_add_(1, chosen, g)
    if score == "sigmoid":
        d = ds * s * (1.0 - s)
    else:
        d = s * (ds - (ds * s).sum(1, keepdim=True))
    return d.to(logits.dtype)


_TANH = math.sqrt(2.0 / math.pi)


def _plain_act(z, act):
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * torch.erfc(-z * math.sqrt(0.5))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(_TANH * (z + 0.044715 * z * z * z)))
    return z


def _plain_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    if act == "gelu":
        return 0.5 * torch.erfc(-z * math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) / math.sqrt(
            2.0 * math.pi)
    u = torch.tanh(_TANH * (z + 0.044715 * z * z * z))
    return 0.5 * (1.0 + u) + 0.5 * z * (1.0 - u * u) * _TANH * (1.0 + 3 * 0.044715 * z * z)


def _plain_logprob(logits, tokens, top):
    x = logits.float()
    m = x.amax(1, keepdim=True)
    d = x - m
    p = torch.exp(d)
    s = p.sum(1, keepdim=True)
    lse = m + s.log()
    given = (tokens >= 0) & (tokens < x.shape[1])
    at = x.gather(1, torch.where(given, tokens, 0)[:, None])
    out = {"logprob": torch.where(given, (at - lse)[:, 0], 0.0),
           "entropy": (s.log() - (p * d).sum(1, keepdim=True) / s)[:, 0], "lse": lse[:, 0]}
    if top:
        ids = []
        place = torch.arange(x.shape[1], device=x.device)
        for _ in range(top):
            best = x.amax(1, keepdim=True)
            ids.append(torch.where(x == best, place, x.shape[1]).amin(1, keepdim=True))
            x = x.scatter(1, ids[-1], -math.inf)
        ids = torch.cat(ids, 1)
        out["top_ids"] = ids.to(torch.int32)
        out["top_logprobs"] = logits.gather(1, ids).float() - lse
    return out


def _plain_logprob_grad(logits, tokens, lse, entropy, dlogprob, dentropy):
    given = (tokens >= 0) & (tokens < logits.shape[1])
    g = torch.where(given, dlogprob, 0.0)[:, None]
    lp = logits.float() - lse[:, None]
    p = torch.exp(lp)
    d = -g * p
    if dentropy is not None:
        d = d - dentropy[:, None] * p * (lp + entropy[:, None])
    d.scatter_add_(1, torch.where(given, tokens, 0)[:, None], g)
    return d.to(logits.dtype)


# ---- the definitions in 64 bits ----------------------------------------------------------


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(state)
    if op == "route_grad":
        return _exact_route_grad(state)
    if op.startswith("gemm"):
        return _exact_gemm(state)
    return _exact_logprob(state) if op == "logprob" else _exact_logprob_grad(state)


def _exact_route(state):
    x = state["logits"].double()
    t, e = x.shape
    s = torch.sigmoid(x) if state["score"] == "sigmoid" else torch.softmax(x, 1)
    c = s if state["bias"] is None else s + state["bias"].double()
    value = x.clone() if state["bias"] is None else c.clone()
    size = e // state["groups"]
    if state["top_groups"] < state["groups"]:
        worth = torch.stack([c[:, g * size:(g + 1) * size].topk(state["group_best"], 1).values.sum(1)
                             for g in range(state["groups"])], 1).cpu()
        for row, w in enumerate(worth.tolist()):
            order = sorted(range(state["groups"]), key=lambda g: (-w[g], g))
            for g in order[state["top_groups"]:]:
                value[row, g * size:(g + 1) * size] = -math.inf
    chosen = torch.argsort(value, dim=1, descending=True, stable=True)[:, :state["k"]]
    # In logarithms: the weights add up to `scale` whatever the scores' size.
    log = torch.log_softmax(x, 1) if state["score"] == "softmax" else -torch.log1p(torch.exp(-x))
    return {"experts": chosen.to(torch.int32),
            "weights": 2.5 * torch.softmax(torch.gather(log, 1, chosen), 1)}


def _exact_route_grad(state):
    x = state["logits"].double().requires_grad_()
    s = torch.sigmoid(x) if state["score"] == "sigmoid" else torch.softmax(x, 1)
    w = torch.gather(s, 1, state["chosen"].long())
    if state["renormalise"]:
        w = w / w.sum(1, keepdim=True)
    (2.5 * w * state["dweights"].double()).sum().backward()
    return x.grad


def _exact_gemm(state):
    act = {"none": lambda z: z, "relu": torch.nn.functional.relu,
           "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
           "gelu_tanh": lambda z: torch.nn.functional.gelu(z, approximate="tanh")}[state["act"]]
    x, w = state["x"].double(), state["w"].double()
    if state["op"] == "gemm_bias_act":
        z = torch.mm(x, w)
        if state["bias"] is not None:
            z += state["bias"].double()
        y = act(z)
        if state["residual"] is not None:
            y = y + state["residual"].double()
        return (y, z) if state["pre"] else y
    dz = state["dy"].double()
    if state["z"] is not None:
        z = state["z"].double().requires_grad_()
        act(z).backward(dz)
        dz = z.grad
    out = {"dx": torch.mm(dz, w.T), "dw": torch.mm(x.T, dz)}
    if state["bias"]:
        out["dbias"] = torch.einsum("tn->n", dz)
    return out


def _pieces(rows):
    """Ranges of rows, few enough at a time for 64-bit copies."""
    return [slice(i, min(i + 256, rows)) for i in range(0, rows, 256)]


def _exact_logprob(state):
    outs = []
    for part in _pieces(state["logits"].shape[0]):
        lp = torch.log_softmax(state["logits"][part].double(), 1)
        lse = torch.logsumexp(state["logits"][part].double(), 1)
        tokens = state["tokens"][part]
        rows = torch.arange(tokens.numel(), device=tokens.device)
        out = {"logprob": torch.where(tokens < 0, 0.0, lp[rows, tokens.clamp(min=0)]),
               "entropy": -torch.einsum("tv,tv->t", lp.exp(), lp), "lse": lse}
        if state["top"]:
            order = torch.argsort(state["logits"][part].float(), dim=1, descending=True,
                                  stable=True)[:, :state["top"]]
            out["top_ids"] = order.to(torch.int32)
            out["top_logprobs"] = torch.gather(lp, 1, order)
        outs.append(out)
    return {k: torch.cat([o[k] for o in outs]) for k in outs[0]}


def _exact_logprob_grad(state):
    # The forward pass's lse and entropy are inputs: they are taken as they are given.
    outs = []
    for part in _pieces(state["logits"].shape[0]):
        lp = state["logits"][part].double() - state["lse"][part].double()[:, None]
        p = lp.exp()
        tokens, g = state["tokens"][part], state["dlogprob"][part].double()
        hot = torch.zeros_like(p)
        rows = torch.arange(tokens.numel(), device=tokens.device)
        hot[rows, tokens.clamp(min=0)] = (tokens >= 0).double()
        d = (hot - p * (tokens >= 0).double()[:, None]) * g[:, None]
        if state["dentropy"] is not None:
            h = state["entropy_of"][part].double()
            d -= state["dentropy"][part].double()[:, None] * p * (lp + h[:, None])
        outs.append(d)
    return torch.cat(outs)
