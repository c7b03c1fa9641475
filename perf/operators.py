"""Measured cases of the grouped operators: the row grouping, the grouped product and its weight
gradient, and low-rank adapters beside a shared projection.

Each case is a dict of plain values with an ``op``:

* ``group_rows``: the stable grouping of ``tokens`` x ``fan`` slots by their group's number (which
  expert, or which adapter, a row goes to);
* ``gemm_grouped``: y[p] = x[rows[p]] w[g] for the rows p of each group g, with w (groups, K, N), or
  (with ``trans``) stored (groups, N, K) as the gradient with respect to x reads it;
* ``gemm_grouped_wgrad``: dw[g] = sum over the rows p of group g of x[rows[p]]^T dy[p];
* ``gemm_lora``: y[t] = x[t] w + scale[g] (x[t] a[g]) b[g], g the adapter of row t (or none).

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
        # One decode step of 37 requests, two experts each: the smallest plan, latency only.
        {"name": "group decode 37x2 of 8", "op": "group_rows", "tokens": 37, "fan": 2, "groups": 8},
        # A prefill or training batch over many small experts.
        {"name": "group batch 16384x8 of 256", "op": "group_rows", "tokens": 16384, "fan": 8,
         "groups": 256},
        # A single token through its two experts: reading two weight matrices is all there is.
        {"name": "experts 1 token bf16", "op": "gemm_grouped", "tokens": 1, "fan": 2, "groups": 8,
         "K": 4096, "N": 4096, "dtype": "bf16", "trans": False, "gather": True},
        # A decode batch: every expert is read for a handful of rows.
        {"name": "experts 64 tokens fp16", "op": "gemm_grouped", "tokens": 64, "fan": 4,
         "groups": 32, "K": 2048, "N": 1024, "dtype": "fp16", "trans": True, "gather": True},
        # A training batch through eight experts, rows fetched through the plan.
        {"name": "experts 8192 tokens bf16", "op": "gemm_grouped", "tokens": 8192, "fan": 2,
         "groups": 8, "K": 4096, "N": 4096, "dtype": "bf16", "trans": False, "gather": True},
        # Single precision at odd sizes, in the direction of the gradient of x.
        {"name": "experts dx 3001 rows fp32", "op": "gemm_grouped", "tokens": 3001, "fan": 1,
         "groups": 5, "K": 1000, "N": 2047, "dtype": "fp32", "trans": True, "gather": False},
        # The weight gradient of the training batch.
        {"name": "dw 4096 tokens bf16", "op": "gemm_grouped_wgrad", "tokens": 4096, "fan": 2,
         "groups": 8, "K": 4096, "N": 4096, "dtype": "bf16", "gather": True},
        # The weight gradient in single precision at odd sizes, many groups with few rows or none.
        {"name": "dw 2047 rows fp32", "op": "gemm_grouped_wgrad", "tokens": 2047, "fan": 1,
         "groups": 33, "K": 1000, "N": 515, "dtype": "fp32", "gather": False},
        # One request with its adapter: the shared weights are all that is read.
        {"name": "adapter 1 token bf16", "op": "gemm_lora", "tokens": 1, "groups": 4, "K": 4096,
         "N": 4096, "rank": 16, "dtype": "bf16", "runs": False},
        # A decode batch in which nearly every request has an adapter of its own.
        {"name": "adapters 64 tokens bf16", "op": "gemm_lora", "tokens": 64, "groups": 64,
         "K": 4096, "N": 4096, "rank": 16, "dtype": "bf16", "runs": False},
        # Prefill: a few requests of many tokens each.
        {"name": "adapters 4096 tokens fp16", "op": "gemm_lora", "tokens": 4096, "groups": 6,
         "K": 4096, "N": 4096, "rank": 64, "dtype": "fp16", "runs": True},
        # Single precision, odd sizes, rows of all adapters mixed.
        {"name": "adapters 257 tokens fp32", "op": "gemm_lora", "tokens": 257, "groups": 7,
         "K": 1000, "N": 2047, "rank": 24, "dtype": "fp32", "runs": False},
    ]


def _between(rng, lo, hi):
    """A size between lo and hi, its logarithm spread evenly; odd ones among them."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A matrix dimension: three in four 1, 1.25 or 1.75 times a power of two, the others odd."""
    v = _between(rng, lo, hi)
    if rng.random() < 0.25:
        return v | 1
    steps = [int(m * 2 ** e) for e in range(6, 13) for m in (1, 1.25, 1.75)]
    return min((s for s in steps if lo <= s <= hi), key=lambda s: abs(math.log(s / v)))


def draw(rng):
    op = rng.choice(["group_rows", "gemm_grouped", "gemm_grouped", "gemm_grouped_wgrad",
                     "gemm_lora", "gemm_lora"])
    most = max(work(c)["flops"] for c in listed())
    while True:
        if op == "group_rows":
            case = {"op": op, "tokens": _between(rng, 1, 16384), "fan": rng.choice([1, 2, 4, 6, 8]),
                    "groups": _between(rng, 4, 256)}
            if case["fan"] > case["groups"]:
                continue
            return case
        case = {"op": op, "tokens": _between(rng, 1, 8192),
                "groups": _between(rng, 2, 64), "K": _width(rng, 64, 4096),
                "N": _width(rng, 64, 4096), "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"])}
        if op == "gemm_lora":
            case["rank"] = rng.choice([8, 16, 20, 32, 64, 100])
            case["runs"] = rng.random() < 0.5
        else:
            case["fan"] = rng.choice([1, 2, 4])
            case["gather"] = rng.random() < 0.5
            if op == "gemm_grouped":
                case["trans"] = rng.random() < 0.5
            if case["fan"] > case["groups"]:
                continue
        w = work(case)
        single = 8 if case["dtype"] == "fp32" else 1   # single precision costs more per operation
        if w["flops"] * single <= most and _weights(case) <= 4096 * 4096 * 8:
            return case


def _weights(case):
    """Weight elements of all groups (and of the shared projection)."""
    K, N = case["K"], case["N"]
    if case["op"] == "gemm_lora":
        return K * N + case["groups"] * case["rank"] * (K + N)
    return case["groups"] * K * N


def _active(slots, groups, fan):
    """Expected number of groups that get a row."""
    return groups * (1.0 - (1.0 - fan / groups) ** (slots // fan))


def work(case):
    op, t, g = case["op"], case["tokens"], case["groups"]
    if op == "group_rows":
        s = t * case["fan"]
        return {"bytes": 4.0 * (s + 3 * s + g + 1), "flops": 0.0}
    size, K, N = _BYTES[case["dtype"]], case["K"], case["N"]
    if op == "gemm_lora":
        r = case["rank"]
        on = _active(t, g, 1)
        return {"bytes": size * (t * K + K * N + on * r * (K + N) + t * N) + 4.0 * t,
                "flops": 2.0 * t * (K * N + r * (K + N))}
    slots = t * case["fan"]
    x_rows = t if case["gather"] else slots
    if op == "gemm_grouped":
        moved = x_rows * K + _active(slots, g, case["fan"]) * K * N + slots * N
    else:
        moved = x_rows * K + slots * N + g * K * N
    return {"bytes": size * moved + 4.0 * (g + 1 + (slots if case["gather"] else 0)),
            "flops": 2.0 * slots * K * N}


def _assign(case, gen):
    """The group of every slot (tokens, fan), each token's all different: the largest of noisy
    scores with some groups more popular than others, as a router's are."""
    t, g = case["tokens"], case["groups"]
    popular = 0.7 * torch.randn(g, device="cuda", generator=gen)
    score = torch.randn(t, g, device="cuda", generator=gen) + popular
    return score.topk(case["fan"], dim=1).indices.to(torch.int32).contiguous()


def _adapters(case, gen):
    """The adapter of every row, -1 (none) for about one row in eight."""
    t, g = case["tokens"], case["groups"]
    if case["runs"]:      # whole requests after one another, an adapter each
        cuts = torch.rand(max(1, min(t, 2 * g)) - 1, device="cuda", generator=gen).mul(t).long()
        run = torch.zeros(t, dtype=torch.long, device="cuda").index_add_(
            0, cuts, torch.ones_like(cuts)).cumsum(0)
        owner = torch.randint(-1, g, (int(run[-1]) + 1,), device="cuda", generator=gen)
        return owner[run].to(torch.int32)
    index = torch.randint(0, g, (t,), device="cuda", generator=gen, dtype=torch.int32)
    if t > 1:
        index[torch.rand(t, device="cuda", generator=gen) < 0.125] = -1
    return index


def _plan(index, groups):
    """(offsets, order): the slots sorted by group, those of no group last."""
    flat = index.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < groups), flat, groups)
    order = torch.argsort(key, stable=True)
    edges = torch.arange(groups + 1, device=key.device)
    offsets = torch.searchsorted(key[order].contiguous(), edges)
    return offsets.to(torch.int32), order.to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, groups = case["op"], case["groups"]
    state = {"op": op, "groups": groups}
    if op == "group_rows":
        state["index"] = _assign(case, gen)
        return state
    dtype, K, N, t = _TYPES[case["dtype"]], case["K"], case["N"], case["tokens"]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, device="cuda", generator=gen) * std).to(dtype)

    if op == "gemm_lora":
        r = case["rank"]
        index = _adapters(case, gen)
        state["offsets"], state["order"] = _plan(index, groups)
        state["x"] = normal(t, K)
        state["w"] = normal(K, N, std=K ** -0.5)
        state["a"] = normal(groups, K, r, std=K ** -0.5)
        state["b"] = normal(groups, r, N, std=0.5 * r ** -0.5)
        state["scale"] = torch.rand(groups, device="cuda", generator=gen) * 1.5 + 0.5
        return state
    offsets, order = _plan(_assign(case, gen), groups)
    slots = t * case["fan"]
    state["offsets"] = offsets
    state["rows"] = order // case["fan"] if case["gather"] else None
    state["most"] = int((offsets[1:] - offsets[:-1]).max())   # of one group, for the plain form
    state["x"] = normal(t if case["gather"] else slots, K)
    if op == "gemm_grouped":
        if case["trans"]:
            state["w"] = normal(groups, N, K, std=K ** -0.5).transpose(1, 2)
        else:
            state["w"] = normal(groups, K, N, std=K ** -0.5)
    else:
        state["dy"] = normal(slots, N)
    return state


def run(state):
    if own:
        return _run_own(state)
    op = state["op"]
    if op == "group_rows":
        return _plain_group(state["index"], state["groups"])
    if op == "gemm_grouped":
        return _plain_grouped(state["x"], state["w"], state["offsets"], state["rows"],
                              state["most"])
    if op == "gemm_grouped_wgrad":
        return _plain_wgrad(state["x"], state["dy"], state["offsets"], state["rows"],
                            state["most"])
    return _plain_lora(state["x"], state["w"], state["a"], state["b"], state["scale"],
                       state["offsets"], state["order"])


def _run_own(state):
    import tiled_matrix_multiply_gb300 as tmm
    op = state["op"]
    if op == "group_rows":
        plan = tmm.group_rows(state["index"], state["groups"])
        return {"offsets": plan.offsets, "order": plan.order, "rows": plan.rows,
                "position": plan.position}
    if op == "gemm_grouped":
        return tmm.gemm_grouped(state["x"], state["w"], state["offsets"], rows=state["rows"])
    if op == "gemm_grouped_wgrad":
        return tmm.gemm_grouped_wgrad(state["x"], state["dy"], state["offsets"],
                                      rows=state["rows"])
    return tmm.gemm_lora(state["x"], state["w"], state["a"], state["b"], state["scale"],
                         state["offsets"], rows=state["order"])


# ---- the plain forms ---------------------------------------------------------------------


def _plain_group(index, groups):
    flat = index.reshape(-1)
    key = torch.where((flat >= 0) & (flat < groups), flat, groups)
    ordered, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(ordered, torch.arange(groups + 1, device=key.device,
                                                       dtype=key.dtype))
    position = torch.empty_like(order)
    position[order] = torch.arange(order.numel(), device=key.device)
    fan = index.shape[1]
    return {"offsets": offsets.to(torch.int32), "order": order.to(torch.int32),
            "rows": (order // fan).to(torch.int32), "position": position.to(torch.int32)}


def _padded(values, offsets, most):
    """The rows of every group, padded with zero rows to `most`: (groups, most, columns), 32 bits."""
    at = offsets[:-1, None] + torch.arange(most, device=values.device)
    inside = at < offsets[1:, None]
    return torch.where(inside[..., None], values[torch.where(inside, at, 0)].float(), 0.0)


def _plain_grouped(x, w, offsets, rows, most):
    if rows is not None:
        x = x[rows]
    y = torch.bmm(_padded(x, offsets, most), w.float())
    p = torch.arange(x.shape[0], device=x.device, dtype=offsets.dtype)
    group = torch.searchsorted(offsets[1:].contiguous(), p, right=True)
    return y[group, p - offsets[group]].to(x.dtype)


def _plain_wgrad(x, dy, offsets, rows, most):
    if rows is not None:
        x = x[rows]
    return torch.bmm(_padded(x, offsets, most).transpose(1, 2),
                     _padded(dy, offsets, most)).to(x.dtype)


def _plain_lora(x, w, a, b, scale, offsets, order):
    groups, k, r = a.shape
    p = torch.arange(x.shape[0], device=x.device, dtype=offsets.dtype)
    owner = torch.empty_like(order)
    owner[order] = torch.searchsorted(offsets[1:].contiguous(), p, right=True).to(order.dtype)
    xf = x.float()
    low = (xf @ a.float().transpose(0, 1).reshape(k, groups * r)).view(-1, groups, r)
    mine = owner[:, None] == torch.arange(groups, device=x.device)
    low = torch.where(mine[..., None], low * scale[:, None], 0.0)
    y = xf @ w.float() + low.view(-1, groups * r) @ b.float().view(groups * r, -1)
    return y.to(x.dtype)


# ---- the definitions in 64 bits ----------------------------------------------------------


def exact(case, seed):
    state = prepare(case, seed)
    op, groups = case["op"], case["groups"]
    if op == "group_rows":
        index = state["index"].reshape(-1).tolist()
        slots = [[] for _ in range(groups)]
        for s, g in enumerate(index):
            slots[g].append(s)
        order = [s for g in slots for s in g]
        offsets, position = [0], [0] * len(order)
        for g in slots:
            offsets.append(offsets[-1] + len(g))
        for p, s in enumerate(order):
            position[s] = p
        return {"offsets": torch.tensor(offsets, dtype=torch.int32),
                "order": torch.tensor(order, dtype=torch.int32),
                "rows": torch.tensor([s // case["fan"] for s in order], dtype=torch.int32),
                "position": torch.tensor(position, dtype=torch.int32)}
    edges = state["offsets"].tolist()
    x = state["x"].double()
    if op == "gemm_lora":
        y = x @ state["w"].double()
        order = state["order"].long()
        for g in range(groups):
            mine = order[edges[g]:edges[g + 1]]
            low = x[mine] @ state["a"][g].double()
            y[mine] += float(state["scale"][g]) * (low @ state["b"][g].double())
        return y
    if state["rows"] is not None:
        x = x[state["rows"].long()]
    if op == "gemm_grouped":
        return torch.cat([x[edges[g]:edges[g + 1]] @ state["w"][g].double()
                          for g in range(groups)])
    dy = state["dy"].double()
    return torch.stack([x[edges[g]:edges[g + 1]].T @ dy[edges[g]:edges[g + 1]]
                        for g in range(groups)])
