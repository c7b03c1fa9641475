"""Operators one after another without a pause, each reading what the one before has just written (and
has perhaps written over what an earlier one read): the results are those of calls waited for."""
import pytest

torch = pytest.importorskip("torch")

import tiled_matrix_multiply_gb300 as tmm  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tiled_matrix_multiply_gb300 import build
    build.build()


def chain(hidden, weights, logits, tokens, wait):
    """Routing, grouped and plain layers and their gradients, and log probabilities of logits that the
    layer writes in place and whose gradient then takes their place."""
    router, experts, w, out, a, b = weights
    r = tmm.route_rows(tmm.gemm_bias_act(hidden, router), 2)
    wait()
    plan = tmm.group_rows(r.experts, experts.shape[0])
    wait()
    y = tmm.gemm_grouped(hidden, experts, plan.offsets, rows=plan.rows)
    wait()
    y = y[:hidden.shape[0]].contiguous()
    z, pre = tmm.gemm_bias_act(y, w, act="gelu", residual=hidden, pre=True)
    wait()
    one = tmm.group_rows(tokens % a.shape[0], a.shape[0])
    wait()
    ranked = tmm.gemm_lora(z, w, a, b, torch.ones(a.shape[0], device="cuda"), one.offsets,
                           rows=one.order)
    wait()
    tmm.gemm_bias_act(z, out, y=logits)
    wait()
    p = tmm.logprob_rows(logits, tokens, top=3)
    wait()
    tmm.logprob_rows_grad(logits, tokens, p.lse, dlogprob=p.entropy, dlogits=logits)
    wait()
    q = tmm.logprob_rows(logits, tokens, top=3)
    wait()
    g = tmm.gemm_bias_act_grad(z, y, w, pre=pre, act="gelu", dbias=True)
    wait()
    return [*r, plan.offsets, plan.order, z, ranked, logits.clone(), *p, *q, *g]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=str)
@pytest.mark.parametrize("T,V", [(3, 4099), (70, 1001), (1300, 513)])
def test_a_chain_without_pauses(dtype, T, V):
    H, E = 136, 8
    gen = torch.Generator().manual_seed(T)

    def rand(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen) * std).to(dtype).cuda()

    weights = (rand(H, E), rand(E, H, H, std=0.1), rand(H, H, std=0.1), rand(H, V, std=0.2),
               rand(4, H, 16, std=0.1), rand(4, 16, H, std=0.1))
    tokens = torch.randint(0, V, (T,), generator=gen).cuda()
    inputs = [rand(T, H) for _ in range(6)]
    logits = torch.empty(T, V, dtype=dtype, device="cuda")
    want = [chain(x, weights, logits, tokens, torch.cuda.synchronize) for x in inputs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [chain(x, weights, logits, tokens, lambda: None) for x in inputs]
    for _ in range(5):
        graph.replay()
        torch.cuda.synchronize()
        for mine, other in zip(got, want):
            assert all(torch.equal(m, o) for m, o in zip(mine, other))
    for _ in range(3):
        eager = [chain(x, weights, logits, tokens, lambda: None) for x in inputs]
        for mine, other in zip(eager, want):
            assert all(torch.equal(m, o) for m, o in zip(mine, other))
    tmm.check_device()
