"""Linear layers at the ends of their types' ranges: what has to pass through fewer bits on its way
must not lose more than those bits."""
import math

import pytest

torch = pytest.importorskip("torch")

import linear_ref as ref  # noqa: E402
import tiled_matrix_multiply_gb300 as tmm  # noqa: E402
from grouped_ref import HALF_STEP, sum_error  # noqa: E402

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]
SMOOTH = ("silu", "gelu", "gelu_tanh")
F16 = torch.float16


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tiled_matrix_multiply_gb300 import build
    build.build()


def normals(seed, *shape, std=1.0):
    gen = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=gen, dtype=torch.float64) * std


def strided(t, ld, offset, fill):
    store = torch.full((offset + t.shape[0] * ld + 8,), fill, dtype=t.dtype, device="cuda")
    view = store[offset:offset + t.shape[0] * ld].view(t.shape[0], ld)[:, :t.shape[1]]
    view.copy_(t)
    return view


def check_half_gradients(dy, x, w, z, kind, got):
    """dz = dy act'(z) is rounded to FP16's eleven bits, and to 2^-39 of the largest |dy| (FP16's
    smallest step beside a largest value of 2^14 and more); the slope's error is linear_ref's."""
    d, zd, xd, wd = dy.double(), z.double(), x.double(), w.double()
    near = zd.abs().clamp(max=13.0)
    slope = ref.slope(zd, kind)
    dz = d * slope
    dz_err = d.abs() * (1 + near) * (3 * near * near + 2 * near + 12) * 2.0 ** -22
    peak = float(d[d.isfinite()].abs().max())
    rounded = dz_err + HALF_STEP[F16] * (dz.abs() + dz_err) + peak * 2.0 ** -39
    size = dz.abs() + rounded
    M, N = dy.shape
    ref.assert_close(got.dx, dz @ wd.T, sum_error(F16, N) * (size @ wd.abs().T)
                     + rounded @ wd.abs().T, "dx")
    ref.assert_close(got.dw, xd.T @ dz, sum_error(F16, M) * (xd.abs().T @ size)
                     + xd.abs().T @ rounded, "dw")
    ref.assert_close(got.dbias, dz.sum(0), dz_err.sum(0)
                     + (M / 8 + 80) * 2.0 ** -24 * dz.abs().sum(0), "dbias")


@pytest.mark.parametrize("kind", SMOOTH)
@pytest.mark.parametrize("M,N,K", [(1, 64, 40), (8, 64, 40), (70, 515, 72), (600, 384, 264)])
def test_half_gradients_whose_dz_is_beyond_the_range(kind, M, N, K):
    """Slopes reach 1.1 and dy 65504; the products of small weights and inputs are finite."""
    dy = torch.where(normals(1, M, N) > 0, 65504.0, -60000.0).to(F16)
    z = (1.4 + 0.9 * (kind == "silu") + normals(2, M, N, std=0.2)).to(F16)
    x, w = normals(3, M, K, std=2.0 ** -9).to(F16), normals(4, K, N, std=2.0 ** -9).to(F16)
    assert bool((dy.double() * ref.slope(z.double(), kind)).abs().max() > 65520)
    g = tmm.gemm_bias_act_grad(dy.cuda(), x.cuda(), w.cuda(), pre=z.cuda(), act=kind, dbias=True)
    check_half_gradients(dy, x, w, z, kind, g)


@pytest.mark.parametrize("kind", SMOOTH)
@pytest.mark.parametrize("size", [2.0 ** -24, 2.0 ** -20, 2.0 ** -16, 2.0 ** -13])
@pytest.mark.parametrize("M,N,K", [(8, 64, 40), (70, 515, 72), (600, 384, 264)])
def test_half_gradients_whose_dz_is_below_the_range(kind, size, M, N, K):
    """Large weights and inputs bring the products of small dz back."""
    dy = normals(1, M, N, std=size).to(F16)
    dy[0, 0] = size
    z = normals(2, M, N, std=2.0).to(F16)
    x, w = normals(3, M, K, std=64.0).to(F16), normals(4, K, N, std=64.0).to(F16)
    g = tmm.gemm_bias_act_grad(dy.cuda(), x.cuda(), w.cuda().t().contiguous().t(), pre=z.cuda(),
                               act=kind, dbias=True)
    check_half_gradients(dy, x, w, z, kind, g)


@pytest.mark.parametrize("extra,offset", [(0, 1), (1, 0), (8, 8), (3, 5)])
def test_half_gradients_of_strided_dy(extra, offset):
    """What lies between the rows has no part in the range."""
    M, N, K = 130, 264, 72
    dy, z = normals(1, M, N, std=2.0 ** -20).to(F16), normals(2, M, N, std=2.0).to(F16)
    x, w = normals(3, M, K, std=64.0).to(F16), normals(4, K, N, std=64.0).to(F16)
    args = x.cuda(), w.cuda()
    given = strided(dy, N + extra, offset, 60000.0)
    g = tmm.gemm_bias_act_grad(given, *args, pre=z.cuda(), act="gelu", dbias=True)
    check_half_gradients(dy, x, w, z, "gelu", g)
    part = tmm.gemm_bias_act_grad(given, None, args[1], pre=z.cuda(), act="gelu", dw=False)
    assert torch.equal(part.dx, g.dx)
    part = tmm.gemm_bias_act_grad(given, args[0], None, pre=z.cuda(), act="gelu", dx=False)
    assert torch.equal(part.dw, g.dw)


def test_half_gradients_with_infinities_and_nothing():
    """An infinity or NaN in dy stays in its row, and the others keep their range; zeros give zeros."""
    M, N, K = 70, 264, 72
    dy, z = normals(1, M, N, std=2.0 ** -20).to(F16), normals(2, M, N).abs().to(F16)
    w = normals(4, K, N, std=64.0).to(F16)
    odd = dy.clone()
    odd[3, 5], odd[9, 7] = math.inf, math.nan
    want = tmm.gemm_bias_act_grad(dy.cuda(), None, w.cuda(), pre=z.cuda(), act="silu", dw=False).dx
    got = tmm.gemm_bias_act_grad(odd.cuda(), None, w.cuda(), pre=z.cuda(), act="silu", dw=False).dx
    rest = [r for r in range(M) if r not in (3, 9)]
    assert torch.equal(got[rest], want[rest])
    assert not bool(got[3].isfinite().any()) and bool(got[9].isnan().all())
    none = tmm.gemm_bias_act_grad(torch.zeros_like(dy).cuda(), None, w.cuda(), pre=z.cuda(),
                                  act="silu", dw=False).dx
    assert not bool(none.any())


def test_half_gradients_in_a_graph_follow_new_sizes_of_dy():
    M, N, K = 70, 264, 72
    z = normals(2, M, N, std=2.0).to(F16).cuda()
    x, w = normals(3, M, K).to(F16).cuda(), normals(4, K, N).to(F16).cuda()
    dy = normals(1, M, N).to(F16).cuda()

    def work():
        return tmm.gemm_bias_act_grad(dy, x, w, pre=z, act="gelu_tanh", dbias=True)

    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work()
    for size in (2.0 ** -18, 2.0 ** 12, 1.0):
        dy.copy_(normals(5, M, N, std=size))
        graph.replay()
        for a, b in zip(got, work()):
            assert torch.equal(a, b)
    tmm.check_device()


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("kind", ("relu",) + SMOOTH)
@pytest.mark.parametrize("M", [4, 40])
def test_slopes_at_infinities(dtype, kind, M):
    """1 and 0, as far out."""
    z = torch.tensor([math.inf, -math.inf, 60000.0, -60000.0]).to(dtype)
    z = z.repeat(M // 4)[:, None].expand(-1, 24).contiguous().cuda()
    dy, one = torch.full((M, 24), 3.0, dtype=dtype), torch.eye(24, dtype=dtype)
    g = tmm.gemm_bias_act_grad(dy.cuda(), None, one.cuda(), pre=z, act=kind, dw=False, dbias=True)
    want = torch.tensor([3.0, 0.0, 3.0, 0.0]).repeat(M // 4)[:, None].expand(-1, 24)
    assert torch.equal(g.dx.float().cpu(), want)
    assert torch.equal(g.dbias.cpu(), want.sum(0))


@pytest.mark.parametrize("kind", ("relu",) + SMOOTH)
def test_half_layer_below_the_range_has_no_gradient(kind):
    """z = -70000 is kept as -inf; y is 0 there, and so is its slope."""
    M, N, K = 40, 72, 16
    x, w = torch.full((M, K), -70.0, dtype=F16).cuda(), torch.full((K, N), 62.5, dtype=F16).cuda()
    y, z = tmm.gemm_bias_act(x, w, act=kind, pre=True)
    assert not bool(y.any()) and bool((z == -math.inf).all())
    g = tmm.gemm_bias_act_grad(torch.ones_like(y), x, w, pre=z, act=kind, dbias=True)
    assert not any(bool(t.any()) for t in g)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("kind", ("relu",) + SMOOTH)
def test_slopes_at_nan_are_nan(dtype, kind):
    z = torch.ones(20, 24, dtype=dtype)
    z[7, 3] = math.nan
    dy, one = torch.ones(20, 24, dtype=dtype), torch.eye(24, dtype=dtype)
    g = tmm.gemm_bias_act_grad(dy.cuda(), None, one.cuda(), pre=z.cuda(), act=kind, dw=False,
                               dbias=True)
    assert bool(g.dx[7].isnan().all()) and bool(g.dbias[3].isnan())
    assert int(g.dx.isnan().sum()) == 24 and int(g.dbias.isnan().sum()) == 1


def test_gelu_in_single_precision():
    """y = max(z, 0) - |z| Phi(-|z|), one term a sum.  Of the tail, in units of 2^-24 of itself: t is off by
    3 (a denominator's half step, and a reciprocal's whole one), which moves t q(t) by 2.4 times that; q's eight
    steps by two of the sum of the terms' sizes, 2.4 q, each, 38; the fit by 0.4; z^2 / 2 by its own
    half step; the exponential by 4 and 3 for its correction; three products by 3.  In all z^2 / 2 + 56.  y is
    rounded once more, and below 2^-126 the exponential's result is 0."""
    z = torch.cat([torch.linspace(-13, 13, 20001), torch.logspace(-20, 0, 500),
                   -torch.logspace(-20, 0, 500)])
    y = tmm.gemm_bias_act(z[:, None].cuda(), torch.ones(1, 24).cuda(), act="gelu").double().cpu()
    zd = z.double()
    tail = 0.5 * torch.erfc(zd.abs() * math.sqrt(0.5))
    want = zd.clamp(min=0) - zd.abs() * tail
    bound = (zd.abs() * tail * (zd * zd / 2 + 56) + want.abs()) * 2.0 ** -24 + 16 * 2.0 ** -126
    off = (y - want[:, None]).abs() / bound[:, None]
    assert float(off.max()) <= 1, float(off.max())
