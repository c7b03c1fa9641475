"""A layer of routed experts with a dense projection, and an output layer: a training step and a
decode step, by the package's operators alone.

    python examples/routed_layer.py [tokens]

Every token goes to four of sixteen experts (chosen by sigmoid scores within the best two of four groups,
with a bias for balance), through two products each; their results, weighted, pass a projection with a
gelu and the layer's input beside it, and the output layer's logits give the log probabilities of the next
tokens.  The loss is their negative sum, and a tenth of the entropies.
"""
from __future__ import annotations

import os
import sys

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import tiled_matrix_multiply_gb300 as tmm

K, GROUPS, TOP = 4, 4, 2
HOW = dict(score="sigmoid", scale=1.5)


def parameters(T=96, D=128, E=16, H=192, V=1001, seed=0):
    gen = torch.Generator().manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen) * std).cuda()
    return {"x": normal(T, D), "router": normal(D, E, std=D ** -0.5),
            "balance": normal(E, std=0.02), "w1": normal(E, D, H, std=D ** -0.5),
            "w2": normal(E, H, D, std=H ** -0.5), "wo": normal(D, D, std=D ** -0.5),
            "bo": normal(D, std=0.1), "head": normal(V, D, std=D ** -0.5),
            "tokens": torch.randint(-1, V, (T,), generator=gen).cuda()}


def forward(p):
    """The logits of the output layer, and what the backward pass needs."""
    x, T = p["x"], p["x"].shape[0]
    logits = tmm.gemm_bias_act(x, p["router"])
    r = tmm.route_rows(logits, K, bias=p["balance"], groups=GROUPS, top_groups=TOP, group_best=2,
                       **HOW)
    plan = tmm.group_rows(r.experts, p["router"].shape[1])
    h = tmm.gemm_grouped(x, p["w1"], plan.offsets, rows=plan.rows)       # (T * K, inner)
    y = tmm.gemm_grouped(h, p["w2"], plan.offsets)                       # (T * K, model)
    by_slot = y[plan.position.long()].view(T, K, -1)
    mixed = (by_slot * r.weights[..., None]).sum(1)
    out, z = tmm.gemm_bias_act(mixed, p["wo"], p["bo"], "gelu", residual=x, pre=True)
    scores = tmm.gemm_bias_act(out, p["head"].t())
    return scores, (logits, r, plan, h, by_slot, mixed, out, z)


def step(p):
    """What the loss is made of, and the gradients of all parameters and of x."""
    x, T = p["x"], p["x"].shape[0]
    scores, (logits, r, plan, h, by_slot, mixed, out, z) = forward(p)
    lp = tmm.logprob_rows(scores, p["tokens"], top=3)
    g = torch.full((T,), -1.0, device=x.device)
    dh = torch.full((T,), 0.1, device=x.device)
    dscores = tmm.logprob_rows_grad(scores, p["tokens"], lp.lse, dlogprob=g, entropy=lp.entropy,
                                    dentropy=dh)
    top = tmm.gemm_bias_act_grad(dscores, out, p["head"].t())
    dense = tmm.gemm_bias_act_grad(top.dx, mixed, p["wo"], pre=z, act="gelu", dbias=True)
    dslot = dense.dx[:, None] * r.weights[..., None]
    dweights = (dense.dx[:, None] * by_slot).sum(2)
    dy = dslot.reshape(T * K, -1)[plan.order.long()].contiguous()
    dhid = tmm.gemm_grouped(dy, p["w2"].transpose(1, 2), plan.offsets)
    dw2 = tmm.gemm_grouped_wgrad(h, dy, plan.offsets)
    dw1 = tmm.gemm_grouped_wgrad(x, dhid, plan.offsets, rows=plan.rows)
    dx_rows = tmm.gemm_grouped(dhid, p["w1"].transpose(1, 2), plan.offsets)
    dlogits = tmm.route_rows_grad(dweights, logits, r.experts, **HOW)
    route = tmm.gemm_bias_act_grad(dlogits, x, p["router"])
    dx = dx_rows[plan.position.long()].view(T, K, -1).sum(1) + route.dx + top.dx
    return {"experts": r.experts, "logprob": lp.logprob, "entropy": lp.entropy,
            "top": lp.top_ids, "x": dx, "router": route.dw, "w1": dw1, "w2": dw2, "wo": dense.dw,
            "bo": dense.dbias, "head": top.dw.t()}


def main():
    T = int(sys.argv[1]) if len(sys.argv) > 1 else 96
    p = parameters(T=T)
    out = step(p)
    print(f"{T} tokens: log probability {float(out['logprob'].sum()):.3f}, "
          f"entropy {float(out['entropy'].mean()):.3f} a token")
    for name in ("router", "w1", "w2", "wo", "bo", "head"):
        print(f"  gradient of {name}: norm {float(out[name].norm()):.4f}")
    p["x"] = p["x"][:1]                    # one token: the alternatives to show
    scores, _ = forward(p)
    best = tmm.logprob_rows(scores, top=5)
    print("  next token:", ", ".join(f"{i} ({v:.2f})" for i, v in zip(
        best.top_ids[0].tolist(), best.top_logprobs[0].tolist())))
    tmm.check_device()


if __name__ == "__main__":
    main()
