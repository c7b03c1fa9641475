"""Routing to experts and log probabilities on the GPU, against their definitions in 64 bits."""
import itertools
import math

import pytest

torch = pytest.importorskip("torch")

import scores_ref as ref  # noqa: E402
import tiled_matrix_multiply_gb300 as tmm  # noqa: E402

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]
INF = math.inf


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tiled_matrix_multiply_gb300 import build
    build.build()


def normals(seed, *shape, std=1.0, dtype=torch.float32):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=gen) * std).to(dtype)


def strided(t, ld, offset=0):
    """The same matrix on the GPU with another row stride, off the start of its allocation."""
    store = torch.full((offset + t.shape[0] * ld + 8,), float("nan"), dtype=t.dtype, device="cuda")
    view = store[offset:offset + t.shape[0] * ld].view(t.shape[0], ld)[:, :t.shape[1]]
    view.copy_(t)
    return view


# ---- routing -------------------------------------------------------------------------------


def check_route(x, k, bias=None, **how):
    r = tmm.route_rows(x.cuda() if not x.is_cuda else x, k,
                       bias=None if bias is None else bias.cuda(), **how)
    x = x.cpu()
    experts, weights = ref.route(x, k, bias, **how)
    assert torch.equal(r.experts.cpu(), experts)
    ref.assert_close(r.weights, weights, ref.weight_bound(x, experts, weights), "weights")
    return r


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (5, 7, 7), (33, 60, 4), (64, 64, 8),
                                   (17, 129, 16), (40, 256, 8), (9, 511, 6), (6, 512, 16)])
def test_route(dtype, score, T, E, k):
    x = normals(T * 1000 + E, T, E, std=1.5, dtype=dtype)
    for renormalise in (True, False):
        check_route(x, k, score=score, renormalise=renormalise, scale=2.5)
    bias = normals(E, E, std=0.1)
    check_route(x, k, bias, score=score)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top_groups", [
    (8, 2, 1), (16, 16, 3), (32, 32, 20), (60, 4, 2), (160, 8, 3), (256, 8, 4), (255, 5, 2),
    (510, 17, 4), (512, 32, 31), (512, 2, 1), (24, 3, 3)])
def test_route_within_groups(dtype, score, E, groups, top_groups):
    x = normals(E * 100 + groups, 21, E, std=1.5, dtype=dtype)
    bias = normals(E, E, std=0.1)
    k = min(8, E // groups * top_groups)
    for best, b in itertools.product((1, 2), (None, bias)):
        check_route(x, k, b, score=score, groups=groups, top_groups=top_groups, group_best=best)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_ties_go_to_the_lower_number(score):
    gen = torch.Generator().manual_seed(3)
    x = torch.randint(-1, 2, (50, 64), generator=gen).float()      # nearly everything ties
    zero = torch.zeros(64)
    for b in (None, zero):
        check_route(x, 8, b, score=score)
        check_route(x, 4, b, score=score, groups=8, top_groups=3, group_best=2)
        check_route(x, 4, b, score=score, groups=8, top_groups=3, group_best=1)
    check_route(torch.cat([-x[:, :32], x[:, 32:] * 0.0], 1) * 0.0, 5, score=score)      # 0 and -0


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top_groups,best", [(1, 1, 1), (8, 4, 1), (8, 4, 2)])
def test_route_scores_closer_than_single_precision_tells(score, groups, top_groups, best):
    """Biases that make c nearly equal: all scores of a row are within 1e-8 of one another."""
    x = normals(11, 30, 64, std=1.0)
    s = ref.scores(x, score)
    for t in range(30):
        bias = (0.9 - s[t]).float()      # c = 0.9 up to the rounding of the bias
        check_route(x[t:t + 1], 6, bias, score=score, groups=groups, top_groups=top_groups,
                    group_best=best)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,k,at", [(64, 1, 6, 0), (64, 1, 6, 5), (256, 8, 8, 3), (256, 8, 8, 7),
                                           (40, 1, 1, 0), (48, 4, 5, 4), (64, 1, 6, (2, 3)),
                                           (64, 1, 6, (5, 6)), (64, 1, 6, (0, 2, 4))])
def test_route_pairs_closer_than_single_precision_tells(score, E, groups, k, at):
    """Scores number `at` and the next of every row are the same up to the rounding of a logit."""
    T = 200
    x, bias = normals(E, T, E, std=1.2), normals(3, E, std=0.05)
    for j in (at,) if isinstance(at, int) else at:
        s = ref.scores(x, score)
        order = (s + bias.double()).argsort(1, descending=True)
        a, b = order[:, j], order[:, j + 1]
        row = torch.arange(T)
        d = bias[a].double() - bias[b].double()
        if score == "sigmoid":
            x[row, b] = torch.logit((s[row, a] + d).clamp(1e-3, 1 - 1e-6)).float()
        else:      # e_b (1 - d) = e_a + d (the sum of all but e_b)
            e = torch.exp(x.double())
            rest = e.sum(1) - e[row, b]
            x[row, b] = torch.log(((e[row, a] + d * rest) / (1 - d)).clamp(min=1e-6)).float()
    check_route(x, k, bias, score=score, groups=groups, top_groups=max(1, groups // 2),
                group_best=min(groups, 2))


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_route_groups_of_equal_sums_go_to_the_lower_number(dtype, bias):
    """Every group has s(l) + s(-l) = 1, of other l."""
    l = normals(3, 300, 8, dtype=torch.float32).abs().to(dtype)
    x = torch.stack([l, -l, torch.full_like(l, -30.0)], 2)
    x[::2] = x[::2].flip(2)
    b = torch.zeros(24, device="cuda") if bias else None
    r = tmm.route_rows(x.view(300, 24).cuda(), 9, bias=b, score="sigmoid", groups=8, top_groups=3,
                       group_best=2)
    assert torch.equal(r.experts.cpu().sort(1).values, torch.arange(9).expand(300, 9).int())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("size", [1.0, 100.0, 5000.0])
def test_route_groups_of_large_biases_that_cancel(score, size):
    """The groups' values are small sums of large c, whose roundings are of the size of the differences."""
    x = normals(11, 500, 32, std=size * 2e-6)
    bias = torch.tensor([size, -size, -4 * size, -5 * size]).repeat(8)
    check_route(x, 2, bias, score=score, groups=8, top_groups=3, group_best=2)
    check_route(x, 5, bias * (1 + torch.arange(32) // 4 % 2), score=score, groups=8, top_groups=3,
                group_best=2)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_masked_experts(dtype, score):
    x = normals(5, 24, 64, std=2.0, dtype=dtype)
    gen = torch.Generator().manual_seed(8)
    x[torch.rand(24, 64, generator=gen) < 0.5] = -INF
    x[3] = -INF                    # a row of padding
    x[4, :] = -INF
    x[4, 17] = 1.0                 # one expert left
    x[5, 8:] = -INF                # one group left
    x[6] = torch.finfo(dtype).min
    x[7, 1:] = torch.finfo(dtype).min
    bias = normals(6, 64, std=0.1)
    bias[::5] = -INF
    for b in (None, bias):
        for r in (True, False):
            check_route(x, 6, b, score=score, renormalise=r)
        for best in (1, 2):
            check_route(x, 6, b, score=score, groups=8, top_groups=2, group_best=best)
    r = tmm.route_rows(x.cuda(), 6, score=score)
    plan = tmm.group_rows(r.experts, 64)                 # slots of no expert come last
    assert int(plan.offsets[-1]) == int((r.experts >= 0).sum())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_scores_below_the_range(score):
    x = normals(7, 16, 32, std=30.0) - 300.0
    check_route(x, 4, score=score)
    check_route(x, 4, score=score, renormalise=False)


def test_route_rows_that_are_not_finite():
    x = normals(9, 4, 64)
    x[0, 5] = float("nan")
    x[1, 6] = INF
    x[2, 7] = float("nan")
    x[2, 9] = -INF
    for score, groups, bias in itertools.product(("softmax", "sigmoid"), (1, 4),
                                                 (None, normals(1, 64, std=0.1).cuda())):
        r = tmm.route_rows(x.cuda(), 8, bias=bias, score=score, groups=groups, top_groups=max(
            1, groups // 2), group_best=min(groups, 2))
        e, w = r.experts.cpu(), r.weights.cpu()
        for row in range(4):
            mine = e[row][e[row] >= 0].tolist()
            assert len(set(mine)) == len(mine) and all(0 <= i < 64 for i in mine)
        assert bool(torch.isfinite(w[3]).all())
        if groups == 1:
            assert bool(w[0].isnan().all() and w[2].isnan().all())
            assert bool(w[1].isnan().all()) == (score == "softmax")


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_nan_in_a_row_reaches_all_its_weights(dtype, score):
    nan = float("nan")
    x = normals(9, 7, 64, dtype=dtype)
    x[0, 5] = nan
    x[1] = nan
    x[2, 3:] = -INF
    x[2, 1] = nan                  # fewer left than are chosen
    x[3, 6] = INF
    x[4, 8:16] = nan               # all of a group
    x[5, 0] -= 40.0                # beside NaN where the bias is -inf, and the lowest group's
    x[5, 63] = nan
    shut = normals(1, 64, std=0.1)
    shut[63] = -INF
    for groups, best, bias, renormalise in itertools.product(
            (1, 8), (1, 2), (None, normals(1, 64, std=0.1), shut), (True, False)):
        r = tmm.route_rows(x.cuda(), 4, bias=None if bias is None else bias.cuda(), score=score,
                           groups=groups, top_groups=max(1, groups // 2), group_best=best,
                           renormalise=renormalise)
        e, w = r.experts.cpu(), r.weights.cpu()
        for row in range(7):
            mine = e[row][e[row] >= 0].tolist()
            assert len(set(mine)) == len(mine) == (3 if row == 2 else 4)
            assert bool((w[row][e[row] < 0] == 0).all())
            bad = row in (0, 1, 2, 4) or (row == 3 and score == "softmax")
            if row == 5 and (bias is not shut or score == "softmax"):
                continue
            got = w[row][e[row] >= 0]
            assert bool(got.isnan().all() if bad else got.isfinite().all()), (row, groups, best)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("ld,offset", [(64, 1), (65, 0), (72, 8), (67, 3)])
def test_route_strides(dtype, ld, offset):
    x = normals(2, 19, 64, std=1.5, dtype=dtype)
    v = strided(x, ld, offset)
    check_route(v, 4, normals(1, 64, std=0.1), score="sigmoid", groups=4, top_groups=2,
                group_best=2)
    r = tmm.route_rows(v, 4)
    g = normals(3, 19, 4).cuda()
    want, size = ref.route_grad(g.cpu(), x, r.experts.cpu(), "softmax", False)
    got = strided(torch.zeros(19, 64, dtype=dtype), ld, offset)
    tmm.route_rows_grad(g, v, r.experts, renormalise=False, dlogits=got)
    # (Not bit for bit what a contiguous matrix gives: a row's sum of 64 exponentials is made in the
    # order of the lanes' shares, whole vectors or single values, and two orders of n - 1 FP32
    # additions of positive terms may differ by 2 (n - 1) half steps.  Either is within the bound of
    # test_route_grad, whose derivation counts 32 + 5 additions.)
    ref.assert_close(got, want, size * (2 * 16 + 100) * ref.STEP + 2.0 ** -140, "dlogits")
    assert bool(v.isfinite().all())


def test_route_many_rows():
    x = normals(4, 16384, 256, std=1.5)
    bias = normals(5, 256, std=0.1)
    r = tmm.route_rows(x.cuda(), 8, bias=bias.cuda(), score="sigmoid", groups=8, top_groups=4,
                       group_best=2)
    c = torch.sigmoid(x.double()) + bias.double()
    best = c.view(-1, 8, 32).topk(2, 2).values.sum(2).topk(4, 1).indices
    open_ = torch.zeros(16384, 8, dtype=torch.bool).scatter_(1, best, True)
    c[~open_.repeat_interleave(32, 1)] = -INF
    assert torch.equal(r.experts.cpu().long(), c.topk(8, 1).indices)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 8, 2), (20, 60, 4), (33, 256, 8), (5, 511, 16),
                                   (4, 512, 3), (6, 100, 6)])
def test_route_grad(dtype, score, renormalise, T, E, k):
    x = normals(T + E, T, E, std=1.5, dtype=dtype)
    x[:, E // 2:E // 2 + E // 8] = -INF
    e = tmm.route_rows(x.cuda(), k, score=score).experts
    if T > 2 and k > 1:
        e[1, 1] = e[1, 0]                        # the same expert twice
        e[2, 0] = -1
        e[2, 1] = E                              # no experts
    g = normals(k, T, k)
    d = tmm.route_rows_grad(g.cuda(), x.cuda(), e, score=score, renormalise=renormalise, scale=1.5)
    want, size = ref.route_grad(g, x, e.cpu(), score, renormalise, 1.5)
    reach = 120.0 if score == "softmax" else 0.0
    reach = min(reach, float((x.double().amax(1, keepdim=True) - x.double())
                             .nan_to_num(0.0, 0.0, 0.0).max()))
    ref.assert_close(d, want, size * (2 * reach + 100) * ref.STEP + 2.0 ** -140, "dlogits")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [True, False])
def test_route_grad_against_differences(score, renormalise):
    x = normals(1, 3, 12, std=1.0).double()
    e, _ = ref.route(x, 4, score=score)
    g = normals(2, 3, 4)
    d = tmm.route_rows_grad(g.cuda(), x.float().cuda(), e.cuda(), score=score,
                            renormalise=renormalise).cpu().double()

    def loss(v):
        w = ref.scores(v, score).gather(1, e.long())
        if renormalise:
            w = w / w.sum(1, keepdim=True)
        return (w * g.double()).sum(1)

    x = x.float().double()
    for c in range(12):
        up, down = x.clone(), x.clone()
        up[:, c] += 1e-4
        down[:, c] -= 1e-4
        slope = (loss(up) - loss(down)) / 2e-4
        assert bool(((slope - d[:, c]).abs() < 1e-6).all())


def test_route_grad_of_nothing_chosen_and_in_place():
    x = normals(1, 4, 32)
    x[2] = -INF
    e = tmm.route_rows(x.cuda(), 4).experts
    g = normals(2, 4, 4).cuda()
    for score, r in itertools.product(("softmax", "sigmoid"), (True, False)):
        d = tmm.route_rows_grad(g, x.cuda(), e, score=score, renormalise=r)
        assert bool((d[2] == 0).all()) and bool(d.isfinite().all())
        v = x.cuda()
        assert tmm.route_rows_grad(g, v, e, score=score, renormalise=r, dlogits=v) is v
        assert torch.equal(v, d)


def test_route_without_tokens():
    x = torch.empty(0, 16, device="cuda")
    r = tmm.route_rows(x, 3)
    assert r.experts.shape == (0, 3) and r.weights.shape == (0, 3)
    assert tmm.route_rows_grad(r.weights, x, r.experts).shape == (0, 16)


# ---- log probabilities ---------------------------------------------------------------------


def check_logprobs(x, tokens=None, top=0, scale=1.0, given=None, times=1):
    """Of logits x, or of `given` on the GPU, which are x's rows as many times."""
    given = x.cuda() if given is None else given
    p = tmm.logprob_rows(given, None if tokens is None else tokens.repeat(times).cuda(), top=top,
                         scale=scale)
    x = x.cpu()
    want, *how = ref.logprobs(x, tokens, top, scale)
    want = {k: v.repeat(times, *[1] * (v.dim() - 1)) for k, v in want.items()}
    how = [v.repeat(times) for v in how]
    lse, lp, ent = ref.logprob_bounds(want, *how, x.shape[1])
    ref.assert_close(p.lse, want["lse"], lse, "lse")
    ref.assert_close(p.entropy, want["entropy"], ent, "entropy")
    if tokens is not None:
        ref.assert_close(p.logprob, want["logprob"],
                         lp + 4 * ref.STEP * want["logprob"].abs().nan_to_num(0.0, 0.0, 0.0),
                         "logprob")
    if top:
        assert torch.equal(p.top_ids.cpu(), want["top_ids"])
        v = want["top_logprobs"]
        ref.assert_close(p.top_logprobs, v,
                         lp[:, None] + 4 * ref.STEP * v.abs().nan_to_num(0.0, 0.0, 0.0), "top")
    return p


def some_tokens(seed, rows, cols, dtype=torch.int64):
    gen = torch.Generator().manual_seed(seed)
    return torch.randint(0, max(cols, 1), (rows,), generator=gen).to(dtype)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("T,V", [(1, 1), (3, 2), (4, 7), (5, 33), (2, 255), (300, 31), (3, 1000),
                                 (2, 4099), (1, 50001), (400, 513), (2, 20000), (1, 131072)])
def test_logprobs(dtype, T, V):
    x = normals(T + V, T, V, std=3.0, dtype=dtype)
    for top in (0, 1, 5, 32):
        check_logprobs(x, some_tokens(V, T, V, torch.int32 if top else torch.int64), top)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("V,ld,offset", [(1000, 1001, 0), (1000, 1003, 1), (999, 1007, 5),
                                         (40000, 40005, 3), (3, 3, 1), (9, 12, 7)])
def test_logprobs_strides(dtype, V, ld, offset):
    x = normals(V, 7, V, std=2.0, dtype=dtype)
    v = strided(x, ld, offset)
    tokens = some_tokens(1, 7, V)
    p = check_logprobs(v, tokens, 6)
    g, h = normals(1, 7).cuda(), normals(2, 7).cuda()
    want = tmm.logprob_rows_grad(x.cuda(), tokens.cuda(), p.lse, dlogprob=g, entropy=p.entropy,
                                 dentropy=h)
    for other, off in ((ld, offset), (ld + 1, offset), (ld, offset + 1)):
        d = strided(torch.zeros(7, V, dtype=dtype), other, off)
        tmm.logprob_rows_grad(v, tokens.cuda(), p.lse, dlogprob=g, entropy=p.entropy, dentropy=h,
                              dlogits=d)
        assert torch.equal(d, want)
    assert torch.equal(v.cpu(), x)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_logprobs_masked_rows(dtype):
    x = normals(5, 9, 3000, std=2.0, dtype=dtype)
    gen = torch.Generator().manual_seed(8)
    x[torch.rand(9, 3000, generator=gen) < 0.5] = -INF
    low = torch.finfo(dtype).min
    x[1] = -INF
    x[2] = -INF
    x[2, 1234] = 3.0
    x[3] = low
    x[4] = low
    x[4, 77] = -2.0
    x[5, 100:] = -INF
    x[5, :100] = low
    x[6, :2990] = -INF
    tokens = torch.tensor([5, 6, 1234, 9, 78, -1, 3000, 2 ** 40, -2 ** 40])
    check_logprobs(x, tokens, 20)
    check_logprobs(x, tokens, 0)


@pytest.mark.parametrize("T", [1, 700])
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_logprobs_rows_that_are_not_finite(dtype, T):
    x = normals(5, T, 9000, dtype=dtype)
    if T > 1:
        x[1, 8999] = float("nan")
        x[2, 4000] = INF
    else:
        x[0, 0] = float("nan")
    p = tmm.logprob_rows(x.cuda(), some_tokens(1, T, 9000).cuda(), top=3)
    bad = [1, 2] if T > 1 else [0]
    for v in (p.logprob, p.entropy, p.lse, p.top_logprobs):
        nan = v.isnan().reshape(T, -1)
        assert bool(nan[bad].all()) and int(nan.any(1).sum()) == len(bad)
    assert bool((p.top_ids[bad] == -1).all())


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("kind", ["rising", "falling", "equal", "ties", "steps"])
def test_alternatives_in_awkward_orders(dtype, kind):
    V = 40000
    i = torch.arange(V).double()
    row = {"rising": i / 700, "falling": -i / 700, "equal": i * 0, "ties": i % 5,
           "steps": (i // 997) % 7}[kind]
    x = torch.stack([row, row.roll(123), -row, row[torch.randperm(
        V, generator=torch.Generator().manual_seed(1))]]).to(dtype)
    check_logprobs(x, some_tokens(2, 4, V), 32)
    many = x.repeat(100, 1)
    p, few = tmm.logprob_rows(many.cuda(), top=32), tmm.logprob_rows(x.cuda(), top=32)
    assert torch.equal(p.top_ids, few.top_ids.repeat(100, 1))


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("V,ld", [(5, 5), (64, 67), (1000, 1000), (3001, 3008), (8001, 8001)])
def test_logprobs_of_many_rows(dtype, V, ld):
    """Rows in numbers, as many as have a warp each and more: the same 26 over and over."""
    T, times, low = 26, 50, torch.finfo(dtype).min
    x = normals(V, T, V, std=2.0, dtype=dtype)
    x[1] = -INF
    x[2] = low
    x[3, 2:] = low
    x[4, 1:] = -INF
    x[5] = 0.25                                   # all alike
    x[6] = (torch.arange(V) % 3).to(dtype)
    x[7] = (torch.arange(V) / 64).to(dtype)
    x[8] = (-torch.arange(V) / 64).to(dtype)
    x[9, : V // 2] = -INF
    tokens = some_tokens(3, T, V)
    tokens[5::7] = -1
    v = strided(x.repeat(times, 1), ld, 1 if ld > V else 0)
    for top in (0, 1, 5, 16, 17, 20, 21, 32):
        # (Not bit for bit the same at every repeat: where a row's first 16-byte boundary lies decides
        # which of its values are added together.)
        check_logprobs(x, tokens, top, given=v, times=times)


@pytest.mark.parametrize("scale", [0.25, 1.0, 3.7])
def test_logprobs_scaled(scale):
    x = normals(3, 6, 5000, std=2.0)
    tokens = some_tokens(3, 6, 5000)
    p = check_logprobs(x, tokens, 4, scale)
    g = normals(4, 6).cuda()
    d = tmm.logprob_rows_grad(x.cuda(), tokens.cuda(), p.lse, dlogprob=g, scale=scale)
    want, err = ref.logprob_grad(x, tokens, p.lse.cpu(), g.cpu(), scale=scale)
    ref.assert_close(d, want, err)


def test_logprobs_without_rows_or_columns():
    p = tmm.logprob_rows(torch.empty(0, 10, device="cuda"), torch.empty(
        0, dtype=torch.int64, device="cuda"), top=2)
    assert p.logprob.shape == (0,) and p.top_ids.shape == (0, 2)
    x = torch.empty(3, 0, device="cuda")
    p = tmm.logprob_rows(x, torch.zeros(3, dtype=torch.int64, device="cuda"), top=2)
    assert p.logprob.tolist() == [0.0] * 3 and p.lse.tolist() == [-INF] * 3
    assert p.entropy.tolist() == [0.0] * 3 and p.top_ids.tolist() == [[-1, -1]] * 3
    assert tmm.logprob_rows_grad(x, None, p.lse).shape == (3, 0)
    assert tmm.logprob_rows(torch.zeros(3, 5, device="cuda")).logprob is None


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("T,V,top", [(1, 1, 1), (5, 33, 4), (300, 50, 0), (4, 4099, 20),
                                     (3, 50001, 32), (2, 9, 3)])
def test_logprob_grad(dtype, T, V, top):
    x = normals(T * V, T, V, std=2.0, dtype=dtype)
    if V > 8:
        x[:, 3:6] = -INF
    if T > 2:
        x[1] = -INF
    tokens = some_tokens(5, T, V)
    if T > 2:
        tokens[2] = -7
    p = tmm.logprob_rows(x.cuda(), tokens.cuda(), top=top)
    g, h = normals(1, T), normals(2, T)
    ids, e = None, None
    if top:
        ids, e = p.top_ids.clone(), normals(3, T, top)
        if top > 2:
            ids[0, 1] = ids[0, 0]                    # the same one twice
            ids[0, 2] = V
    for use_g, use_h, use_e in itertools.product((True, False), repeat=3):
        if use_e and not top:
            continue
        how = dict(dlogprob=g if use_g else None, dentropy=h if use_h else None,
                   entropy=p.entropy.cpu() if use_h else None,
                   top_ids=ids.cpu() if use_e else None, dtop=e if use_e else None)
        d = tmm.logprob_rows_grad(x.cuda(), tokens.cuda(), p.lse, **{
            k: None if v is None else v.cuda() for k, v in how.items()})
        want, err = ref.logprob_grad(x, tokens, p.lse.cpu(), **how)
        ref.assert_close(d, want, err, f"{use_g} {use_h} {use_e}")


def test_logprob_grad_against_differences():
    x = normals(1, 4, 9).double()
    tokens = torch.tensor([0, 8, -1, 3])
    p = tmm.logprob_rows(x.float().cuda(), tokens.cuda(), top=3)
    g, h, e = normals(1, 4), normals(2, 4), normals(3, 4, 3)
    d = tmm.logprob_rows_grad(x.float().cuda(), tokens.cuda(), p.lse, g.cuda(), p.entropy, h.cuda(),
                              p.top_ids, e.cuda()).cpu().double()
    x = x.float().double()
    ids = p.top_ids.cpu().long()

    def loss(v):
        lp = torch.log_softmax(v, 1)
        own = torch.where(tokens < 0, 0.0, lp.gather(1, tokens.clamp(min=0)[:, None])[:, 0])
        return (own * g.double() - (lp.exp() * lp).sum(1) * h.double()
                + (lp.gather(1, ids) * e.double()).sum(1))

    for c in range(9):
        up, down = x.clone(), x.clone()
        up[:, c] += 1e-4
        down[:, c] -= 1e-4
        slope = (loss(up) - loss(down)) / 2e-4
        assert bool(((slope - d[:, c]).abs() < 2e-6).all())


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("V", [1000, 30001])
def test_logprob_grad_in_place(dtype, V):
    x = normals(6, 12, V, dtype=dtype).cuda()
    tokens = some_tokens(1, 12, V).cuda()
    p = tmm.logprob_rows(x, tokens, top=4)
    how = dict(dlogprob=normals(1, 12).cuda(), entropy=p.entropy, dentropy=normals(2, 12).cuda(),
               top_ids=p.top_ids, dtop=normals(3, 12, 4).cuda())
    d = tmm.logprob_rows_grad(x, tokens, p.lse, **how)
    assert tmm.logprob_rows_grad(x, tokens, p.lse, dlogits=x, **how) is x
    assert torch.equal(x, d)


def test_logprob_rows_past_two_billion_values():
    """Row offsets beyond 32 bits."""
    rows, V = 9000, 240001
    x = torch.zeros(rows, V, dtype=torch.bfloat16, device="cuda")
    x[-1, 5] = 4.0
    tokens = torch.full((rows,), 5, device="cuda")
    p = tmm.logprob_rows(x, tokens, top=1)
    assert p.top_ids[-1].item() == 5
    want = 4.0 - math.log(V - 1 + math.exp(4.0))
    assert abs(p.logprob[-1].item() - want) < 1e-4
    assert abs(p.logprob[0].item() + math.log(V)) < 1e-4
    tmm.logprob_rows_grad(x, tokens, p.lse, dlogprob=torch.ones(rows, device="cuda"), dlogits=x)
    assert abs(x[-1, 5].item() - (1 - math.exp(want))) < 4e-3


# ---- both ----------------------------------------------------------------------------------


def test_scores_on_another_stream_and_in_a_graph():
    x = normals(1, 64, 128, std=1.5).cuda()
    y = normals(2, 16, 30001, std=2.0).cuda()
    tokens = some_tokens(2, 16, 30001).cuda()
    gw, gl = normals(3, 64, 4).cuda(), normals(4, 16).cuda()

    def work():
        r = tmm.route_rows(x, 4, score="sigmoid", groups=4, top_groups=2, group_best=2)
        d = tmm.route_rows_grad(gw, x, r.experts, score="sigmoid")
        p = tmm.logprob_rows(y, tokens, top=7)
        e = tmm.logprob_rows_grad(y, tokens, p.lse, dlogprob=gl)
        return (*r, d, *p, e)

    want = work()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    r = tmm.route_rows(x, 4, score="sigmoid", groups=4, top_groups=2, group_best=2, stream=s)
    p = tmm.logprob_rows(y, tokens, top=7, stream=s)
    s.synchronize()
    assert torch.equal(r.experts, want[0]) and torch.equal(p.lse, want[5])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work()
    x.copy_(normals(11, 64, 128, std=1.5))
    y.copy_(normals(12, 16, 30001, std=2.0))
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, work()):
        assert torch.equal(a, b)


def test_scores_calls_at_once():
    """The same calls on several streams give the same bits."""
    y = normals(2, 8, 60000, std=2.0).cuda()
    want = tmm.logprob_rows(y, top=9)
    streams = [torch.cuda.Stream() for _ in range(6)]
    got = []
    for _ in range(4):
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
            got.append(tmm.logprob_rows(y, top=9, stream=s))
    torch.cuda.synchronize()
    for p in got:
        for a, b in zip(p[1:], want[1:]):
            assert torch.equal(a, b)
