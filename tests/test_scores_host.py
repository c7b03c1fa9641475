"""Routing and log probabilities on the host: refusals before any CUDA call (CPU only; no compute
call is made)."""
import math

import pytest

torch = pytest.importorskip("torch")

import scores_ref as ref  # noqa: E402
from tiled_matrix_multiply_gb300 import _abi, build  # noqa: E402

FAKE = 0x7F0000001000          # never dereferenced: every case fails validation first
FAR = [FAKE + (i << 40) for i in range(12)]
BAD, ALIAS = _abi.TMM_ERR_INVALID_ARG, _abi.TMM_ERR_ALIAS


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _abi.load()


def args(defaults, change):
    a = dict(defaults)
    assert not set(change) - set(a)
    a.update(change)
    return list(a.values())


ROUTE = dict(dtype=_abi.TMM_BF16, tokens=16, experts=64, logits=FAR[0], ld=64, bias=FAR[1], score=0,
             groups=8, top_groups=4, group_best=2, k=8, renormalise=1, scale=1.0, chosen=FAR[2],
             weights=FAR[3], stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=3), BAD), (dict(tokens=-1), BAD), (dict(tokens=1 << 29), BAD),
    (dict(experts=0, ld=1), BAD), (dict(experts=513, ld=513), BAD), (dict(ld=63), BAD),
    (dict(ld=1 << 60), BAD), (dict(logits=0), BAD), (dict(logits=FAR[0] + 1), BAD),
    (dict(bias=FAR[1] + 2), BAD), (dict(score=2), BAD), (dict(groups=0), BAD),
    (dict(groups=64), BAD), (dict(groups=7), BAD), (dict(top_groups=0), BAD),
    (dict(top_groups=9), BAD), (dict(group_best=0), BAD), (dict(group_best=3), BAD),
    (dict(k=0), BAD), (dict(k=17), BAD), (dict(top_groups=1, k=9), BAD), (dict(renormalise=2), BAD),
    (dict(scale=math.nan), BAD), (dict(scale=math.inf), BAD), (dict(chosen=0), BAD),
    (dict(weights=0), BAD), (dict(weights=FAR[3] + 2), BAD),
    (dict(chosen=FAR[0] + 64), ALIAS), (dict(weights=FAR[2] + 8), ALIAS),
    (dict(weights=FAR[1]), ALIAS)])
def test_route_refusals(lib, change, status):
    assert lib.route_rows(*args(ROUTE, change)) == status
    assert lib.tmm_last_error_string().decode()


ROUTE_GRAD = dict(dtype=_abi.TMM_F32, tokens=16, experts=64, k=8, dweights=FAR[0], logits=FAR[1],
                  ld=64, chosen=FAR[2], score=1, renormalise=1, scale=1.0, dlogits=FAR[3], ldd=64,
                  stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=-1), BAD), (dict(k=0), BAD), (dict(k=17), BAD), (dict(k=9, experts=8), BAD),
    (dict(ld=63), BAD), (dict(ldd=63), BAD), (dict(dweights=0), BAD), (dict(logits=0), BAD),
    (dict(chosen=0), BAD), (dict(dlogits=0), BAD), (dict(dlogits=FAR[3] + 2), BAD),
    (dict(score=-1), BAD), (dict(scale=math.inf), BAD),
    (dict(dlogits=FAR[1], ldd=65), ALIAS), (dict(dlogits=FAR[0]), ALIAS),
    (dict(dlogits=FAR[2]), ALIAS)])
def test_route_grad_refusals(lib, change, status):
    assert lib.route_rows_grad(*args(ROUTE_GRAD, change)) == status
    assert lib.tmm_last_error_string().decode()


LOGPROB = dict(dtype=_abi.TMM_F16, rows=16, cols=1000, logits=FAR[0], ld=1000, scale=1.0,
               tokens=FAR[1], token_bits=64, top=5, logprob=FAR[2], entropy=FAR[3], lse=FAR[4],
               top_ids=FAR[5], top_logprobs=FAR[6], stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=7), BAD), (dict(rows=-1), BAD), (dict(cols=1 << 29, ld=1 << 29), BAD),
    (dict(ld=999), BAD), (dict(logits=0), BAD), (dict(logits=FAR[0] + 1), BAD),
    (dict(scale=0.0), BAD), (dict(scale=-1.0), BAD), (dict(scale=math.nan), BAD),
    (dict(token_bits=16), BAD), (dict(tokens=FAR[1] + 4), BAD), (dict(top=-1), BAD),
    (dict(top=33), BAD), (dict(tokens=0), BAD), (dict(logprob=0), BAD), (dict(entropy=0), BAD),
    (dict(lse=0), BAD), (dict(top_ids=0), BAD), (dict(top_logprobs=FAR[6] + 1), BAD),
    (dict(lse=FAR[0] + 4), ALIAS), (dict(entropy=FAR[4] + 4), ALIAS), (dict(top_ids=FAR[1]), ALIAS)])
def test_logprob_refusals(lib, change, status):
    assert lib.logprob_rows(*args(LOGPROB, change)) == status
    assert lib.tmm_last_error_string().decode()


LOGPROB_GRAD = dict(dtype=_abi.TMM_F32, rows=16, cols=1000, logits=FAR[0], ld=1000, scale=1.0,
                    lse=FAR[1], tokens=FAR[2], token_bits=32, dlogprob=FAR[3], entropy=FAR[4],
                    dentropy=FAR[5], top=4, top_ids=FAR[6], dtop=FAR[7], dlogits=FAR[8], ldd=1000,
                    stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=7), BAD), (dict(ld=1), BAD), (dict(ldd=1), BAD), (dict(lse=0), BAD),
    (dict(tokens=0), BAD), (dict(entropy=0), BAD), (dict(top_ids=0), BAD), (dict(dtop=0), BAD),
    (dict(dlogits=0), BAD), (dict(scale=0.0), BAD), (dict(top=40), BAD),
    (dict(dlogprob=FAR[3] + 2), BAD), (dict(dlogits=FAR[0], ldd=1001), ALIAS),
    (dict(dlogits=FAR[0] + 4000), ALIAS), (dict(dlogits=FAR[1]), ALIAS),
    (dict(dlogits=FAR[7]), ALIAS)])
def test_logprob_grad_refusals(lib, change, status):
    assert lib.logprob_rows_grad(*args(LOGPROB_GRAD, change)) == status
    assert lib.tmm_last_error_string().decode()


def test_nothing_to_do_needs_no_device(lib):
    assert lib.route_rows(*args(ROUTE, dict(tokens=0))) == _abi.TMM_OK
    assert lib.route_rows_grad(*args(ROUTE_GRAD, dict(tokens=0))) == _abi.TMM_OK
    assert lib.logprob_rows(*args(LOGPROB, dict(rows=0))) == _abi.TMM_OK
    assert lib.logprob_rows_grad(*args(LOGPROB_GRAD, dict(rows=0))) == _abi.TMM_OK
    assert lib.logprob_rows_grad(*args(LOGPROB_GRAD, dict(cols=0))) == _abi.TMM_OK


def test_python_refuses_host_tensors_and_wrong_types():
    import tiled_matrix_multiply_gb300 as tmm
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        tmm.route_rows(x, 2)
    with pytest.raises(TypeError):
        tmm.route_rows(x.double(), 2)
    with pytest.raises(ValueError):
        tmm.logprob_rows(x, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(TypeError):
        tmm.logprob_rows([1.0])


def test_the_definitions_in_64_bits():
    """The reference against torch's own functions."""
    gen = torch.Generator().manual_seed(1)
    x = torch.randn(5, 12, generator=gen, dtype=torch.float64)
    e, w = ref.route(x, 3)
    v, i = torch.softmax(x, 1).topk(3, 1)
    assert torch.equal(e.long(), i)
    assert torch.allclose(w, v / v.sum(1, keepdim=True), rtol=1e-12)
    tokens = torch.tensor([0, 3, -1, 12, 5])
    out, *_ = ref.logprobs(x, tokens, 2)
    lp = torch.log_softmax(x, 1)
    assert torch.allclose(out["lse"], torch.logsumexp(x, 1))
    assert torch.allclose(out["entropy"], -(lp * lp.exp()).sum(1))
    assert torch.allclose(out["logprob"][[0, 1, 4]], lp[[0, 1, 4], [0, 3, 5]])
    assert out["logprob"][2:4].tolist() == [0.0, 0.0]
    assert torch.equal(out["top_ids"].long(), x.topk(2, 1).indices)
    leaf = x.clone().requires_grad_()
    lp = torch.log_softmax(leaf, 1)
    g = torch.randn(5, generator=gen, dtype=torch.float64)
    (lp[[0, 1, 4], [0, 3, 5]] * g[[0, 1, 4]]).sum().backward()
    d, _ = ref.logprob_grad(x, tokens, out["lse"], dlogprob=g)
    assert torch.allclose(d, leaf.grad, atol=1e-12)
    for score, renormalise in (("softmax", True), ("softmax", False), ("sigmoid", True),
                               ("sigmoid", False)):
        leaf = x.clone().requires_grad_()
        s = torch.sigmoid(leaf) if score == "sigmoid" else torch.softmax(leaf, 1)
        w = s.gather(1, e.long())
        if renormalise:
            w = w / w.sum(1, keepdim=True)
        dw = torch.randn(5, 3, generator=gen, dtype=torch.float64)
        (w * dw).sum().backward()
        d, _ = ref.route_grad(dw, x, e, score, renormalise)
        assert torch.allclose(d, leaf.grad, atol=1e-12)
