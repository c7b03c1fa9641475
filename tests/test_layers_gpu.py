"""A run of the operators together, as a model uses them: a layer of routed experts with a dense
projection, and an output layer whose log probabilities are learned; forward and backward against
autograd in 64 bits on the same (rounded) values, and a step captured into a graph."""
import pathlib
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

import tiled_matrix_multiply_gb300 as tmm  # noqa: E402
import routed_layer as ex  # noqa: E402
from routed_layer import GROUPS, K, TOP, parameters, step  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tiled_matrix_multiply_gb300 import build
    build.build()


def reference(p, experts):
    """The same from the formulas by autograd in 64 bits, with the experts chosen."""
    q = {k: v.double().cpu().requires_grad_() for k, v in p.items() if k != "tokens"}
    tokens, e = p["tokens"].cpu(), experts.long().cpu()
    x = q["x"]
    s = torch.sigmoid(x @ q["router"])
    w = s.gather(1, e)
    w = 1.5 * w / w.sum(1, keepdim=True)
    y = torch.einsum("td,tkdh->tkh", x, q["w1"][e])
    y = torch.einsum("tkh,tkhd->tkd", y, q["w2"][e])
    mixed = (y * w[..., None]).sum(1)
    out = torch.nn.functional.gelu(mixed @ q["wo"] + q["bo"]) + x
    scores = out @ q["head"].T
    lp = torch.log_softmax(scores, 1)
    own = torch.where(tokens < 0, 0.0, lp.gather(1, tokens.clamp(min=0)[:, None])[:, 0])
    entropy = -(lp * lp.exp()).sum(1)
    (-own.sum() + 0.1 * entropy.sum()).backward()
    c = torch.sigmoid(x @ q["router"]) + q["balance"]
    best = c.detach().view(-1, GROUPS, c.shape[1] // GROUPS).topk(2, 2).values.sum(2)
    open_ = torch.zeros_like(best).scatter_(1, best.topk(TOP, 1).indices, 1.0)
    shut = open_.repeat_interleave(c.shape[1] // GROUPS, 1) == 0
    chosen = c.detach().masked_fill(shut, -1.0).topk(K, 1).indices
    out = {"experts": chosen.int(), "logprob": own.detach(), "entropy": entropy.detach(),
           "top": scores.detach().topk(3, 1).indices.int()}
    out.update({k: q[k].grad for k in ("x", "router", "w1", "w2", "wo", "bo", "head")})
    return out


def test_a_step_of_experts_a_projection_and_an_output_layer():
    p = parameters()
    got = step(p)
    want = reference(p, got["experts"])
    assert torch.equal(got["experts"].cpu(), want["experts"])
    assert torch.equal(got["top"].cpu(), want["top"])
    for name in ("logprob", "entropy", "x", "router", "w1", "w2", "wo", "bo", "head"):
        a, b = got[name].double().cpu(), want[name]
        # Six FP32 operators after one another, each within 2^-20 of its result's norm (what the
        # header says of a product), and linear in what it is given.
        assert float((a - b).norm() / b.norm()) < 6 * 2.0 ** -20, name
    tmm.check_device()


def test_a_step_replayed_from_a_graph():
    p = parameters()
    step(p)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(p)
    other = parameters(seed=5)
    for k in p:
        p[k].copy_(other[k])
    graph.replay()
    torch.cuda.synchronize()
    want = step(p)
    for k in got:
        assert torch.equal(got[k], want[k]), k


@pytest.mark.parametrize("T", [1, 3])
def test_single_tokens(T):
    """The forward pass of a decode step gives the batch's results, row by row."""
    p = parameters()
    logits = tmm.gemm_bias_act(p["x"], p["router"])
    r = tmm.route_rows(logits, K, score="sigmoid")
    lp = tmm.logprob_rows(logits, top=2)
    for t in range(0, 12, T):
        rows = slice(t, t + T)
        few = tmm.gemm_bias_act(p["x"][rows], p["router"])
        assert float((few - logits[rows]).abs().max()) < 1e-5
        one = tmm.route_rows(logits[rows], K, score="sigmoid")
        assert torch.equal(one.experts, r.experts[rows]) and torch.equal(one.weights,
                                                                         r.weights[rows])
        assert torch.equal(tmm.logprob_rows(logits[rows], top=2).top_ids, lp.top_ids[rows])


FIRST = """
import torch, tiled_matrix_multiply_gb300 as tmm
x, w = torch.ones(200, 64, device="cuda"), torch.ones(64, 96, device="cuda")
tokens = torch.zeros(200, dtype=torch.int64, device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    r = tmm.route_rows(x, 4)
    few = tmm.gemm_bias_act(x[:3], w)
    y, z = tmm.gemm_bias_act(x.half(), w.half(), act="relu", pre=True)
    g = tmm.gemm_bias_act_grad(y, x.half(), w.half(), pre=z, act="relu", dbias=True)
    p = tmm.logprob_rows(x, tokens, top=2)
graph.replay()
torch.cuda.synchronize()
tmm.check_device()
assert r.experts[0].tolist() == [0, 1, 2, 3] and bool((few == 64).all()) and bool((y == 64).all())
assert bool((g.dx == 64 * 96).all()) and bool((g.dbias == 64 * 200).all())
assert p.top_ids[0].tolist() == [0, 1]
"""


def test_first_calls_of_a_process_may_be_captured():
    subprocess.run([sys.executable, "-c", FIRST], check=True, timeout=300,
                   cwd=pathlib.Path(tmm.__file__).parents[1])


def test_the_example_runs(capsys, monkeypatch):
    monkeypatch.setattr("sys.argv", ["routed_layer.py", "33"])
    ex.main()
    assert "33 tokens" in capsys.readouterr().out
