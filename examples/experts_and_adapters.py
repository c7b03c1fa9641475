"""The grouped operators as a model uses them: an expert layer's training step, and a decode step
through a projection with an adapter per request.

    python examples/experts_and_adapters.py [tokens]

The expert layer sends every token through two of eight experts, two products each with a
squared-ReLU between, and adds their results up with the router's weights.  Its backward pass is
made of the same operators: the gradient of a grouped product's rows is the product with the
transposed matrices, that of its matrices gemm_grouped_wgrad.
"""
from __future__ import annotations

import os
import sys

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import tiled_matrix_multiply_gb300 as tmm


def route(logits, fan):
    """(weights, plan): the softmax of every token's `fan` largest logits, and their grouping."""
    top, experts = logits.topk(fan, dim=1)
    weights = tmm.softmax_rows_f32(top.float().contiguous())
    return weights, tmm.group_rows(experts, logits.shape[1])


def experts_forward(x, w1, w2, logits, fan=2):
    """y (tokens, model) and what the backward pass needs."""
    weights, plan = route(logits, fan)
    h = tmm.gemm_grouped(x, w1, plan.offsets, rows=plan.rows)           # (tokens * fan, inner)
    a = torch.relu(h).square()
    z = tmm.gemm_grouped(a, w2, plan.offsets)                           # (tokens * fan, model)
    mine = z[plan.position.view(-1, fan)]                               # (tokens, fan, model)
    y = (mine.float() * weights[..., None]).sum(1).to(x.dtype)
    return y, (x, w1, w2, weights, plan, h, a, mine)


def experts_backward(dy, saved):
    """(dx, dw1, dw2, dlogits of the chosen experts) for the gradient dy of y."""
    x, w1, w2, weights, plan, h, a, mine = saved
    fan = weights.shape[1]
    dweights = (mine.float() * dy.float()[:, None]).sum(2)
    dlogits = weights * (dweights - (weights * dweights).sum(1, keepdim=True))
    token_weight = weights.reshape(-1)[plan.order.long()]
    dz = (dy[plan.rows.long()].float() * token_weight[:, None]).to(x.dtype)
    dw2 = tmm.gemm_grouped_wgrad(a, dz, plan.offsets)
    da = tmm.gemm_grouped(dz, w2.transpose(1, 2), plan.offsets)
    dh = (da.float() * 2.0 * torch.relu(h.float())).to(x.dtype)
    dw1 = tmm.gemm_grouped_wgrad(x, dh, plan.offsets, rows=plan.rows)
    dxs = tmm.gemm_grouped(dh, w1.transpose(1, 2), plan.offsets)
    dx = dxs[plan.position.view(-1, fan)].float().sum(1).to(x.dtype)
    return dx, dw1, dw2, dlogits


def adapters_step(x, w, a, b, scale, adapter):
    """One projection of a batch of requests, row t with adapter adapter[t] (-1: none)."""
    plan = tmm.group_rows(adapter, a.shape[0])
    return tmm.gemm_lora(x, w, a, b, scale, plan.offsets, rows=plan.order)


def main(tokens=2048, model=1024, inner=2048, experts=8, dtype=torch.bfloat16):
    gen = torch.Generator(device="cuda").manual_seed(0)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, device="cuda", generator=gen) * std).to(dtype)

    x = normal(tokens, model)
    w1, w2 = normal(experts, model, inner, std=model ** -0.5), \
        normal(experts, inner, model, std=inner ** -0.5)
    logits = torch.randn(tokens, experts, device="cuda", generator=gen)
    y, saved = experts_forward(x, w1, w2, logits)
    dx, dw1, dw2, dlogits = experts_backward(normal(tokens, model), saved)
    requests, rank = min(tokens, 32), 16
    adapter = torch.randint(-1, 6, (requests,), device="cuda", generator=gen)
    z = adapters_step(x[:requests], w1[0], normal(6, model, rank, std=model ** -0.5),
                      normal(6, rank, inner, std=rank ** -0.5), torch.ones(6, device="cuda"),
                      adapter)
    tmm.check_device()
    return {"y": y, "dx": dx, "dw1": dw1, "dw2": dw2, "dlogits": dlogits, "adapters": z}


if __name__ == "__main__":
    for name, t in main(int(sys.argv[1]) if len(sys.argv) > 1 else 2048).items():
        print(f"{name:9s} {str(tuple(t.shape)):22s} norm {t.float().norm().item():.4f}")
