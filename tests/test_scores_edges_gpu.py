"""Rows of scores with NaN and infinities where no result seems to need them."""
import itertools
import math

import pytest

torch = pytest.importorskip("torch")

import tiled_matrix_multiply_gb300 as tmm  # noqa: E402

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]
INF, NAN = math.inf, math.nan


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tiled_matrix_multiply_gb300 import build
    build.build()


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("odd", [NAN, INF])
@pytest.mark.parametrize("E,shut", [(64, 63), (64, 0), (60, 17), (512, 300)])
def test_route_odd_logits_of_experts_shut_by_their_bias(dtype, odd, E, shut):
    """The softmax is over all experts, so that its scores are NaN; a sigmoid is the expert's own."""
    gen = torch.Generator().manual_seed(E + shut)
    x = torch.randn(5, E, generator=gen).to(dtype)
    x[::2, shut] = odd
    bias = torch.randn(E, generator=gen) * 0.1
    bias[shut] = -INF
    clean = x.clone()
    clean[:, shut] = 0.0
    for groups, best, renormalise in itertools.product((1, 4), (1, 2), (True, False)):
        how = dict(bias=bias.cuda(), groups=groups, top_groups=max(1, groups // 2),
                   group_best=best, renormalise=renormalise)
        r = tmm.route_rows(x.cuda(), 4, score="softmax", **how)
        assert bool(r.weights[::2].isnan().all()), (groups, best, renormalise)
        assert bool(r.weights[1::2].isfinite().all())
        for row in r.experts.tolist():
            assert len(set(row)) == 4 and shut not in row and all(0 <= e < E for e in row)
        r = tmm.route_rows(x.cuda(), 4, score="sigmoid", **how)
        want = tmm.route_rows(clean.cuda(), 4, score="sigmoid", **how)
        assert torch.equal(r.experts, want.experts) and torch.equal(r.weights, want.weights)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("T,V", [(3, 9), (3, 9000), (1300, 513)])
def test_padding_in_rows_that_are_not_finite(dtype, T, V):
    """A padding token's log probability is 0 whatever its row's logits; the row's other results are NaN."""
    x = torch.randn(T, V, generator=torch.Generator().manual_seed(1)).to(dtype)
    x[0, V // 2], x[1, V - 1] = NAN, INF
    tokens = torch.zeros(T, dtype=torch.int64)
    tokens[0], tokens[1] = -100, V
    for top in (0, 3):
        p = tmm.logprob_rows(x.cuda(), tokens.cuda(), top=top)
        assert p.logprob[:2].tolist() == [0.0, 0.0] and bool(p.logprob[2:].isfinite().all())
        assert bool(p.lse[:2].isnan().all() and p.entropy[:2].isnan().all())
        if top:
            assert bool(p.top_logprobs[:2].isnan().all()) and bool((p.top_ids[:2] == -1).all())
    # Without a gradient of their own such rows get zeros.
    g = torch.ones(T, device="cuda")
    d = tmm.logprob_rows_grad(x.cuda(), tokens.cuda(), p.lse, dlogprob=g)
    assert not bool(d[:2].any()) and bool(d.isfinite().all())
