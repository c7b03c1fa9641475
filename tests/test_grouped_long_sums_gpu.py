"""Grouped products whose sums are long: sums leave tensor memory for FP32 registers every few
thousand terms, so that the error of an addition there (not rounded to nearest) does not add up."""
import pytest

torch = pytest.importorskip("torch")

import grouped_ref as ref  # noqa: E402
import tiled_matrix_multiply_gb300 as tmm  # noqa: E402

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]
TAKEN = 8192                # terms of a sum in tensor memory
TAKEN_FP32 = 128            # of a sum of FP32 products, leading or lower parts


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tiled_matrix_multiply_gb300 import build
    build.build()


def ints(gen, *shape, top=1):
    return torch.randint(-top, top + 1, shape, generator=gen).double()


def offsets_of(sizes, first=0):
    return torch.tensor([first] + sizes).cumsum(0).to(torch.int32)


def sums_within(got, want, terms):
    """Sums of positive terms: at most TAKEN of them added in tensor memory, 16 at a time (see
    grouped_ref.sum_error), then one FP32 addition for every TAKEN; rounded once."""
    half = ref.HALF_STEP[got.dtype]
    bound = (TAKEN / 16 + 2) * 2.0 ** -22 + (terms / TAKEN + 10) * 2.0 ** -24
    err = ((got.double() - want) / want).abs().max().item()
    assert err <= half * (1 + bound) + bound, (err, half, bound)


@pytest.mark.parametrize("dtype", TYPES[:2], ids=str)
@pytest.mark.parametrize("K,N,rows", [(130, 256, 2 ** 19 + 77), (60, 100, 2 ** 22 + 5)])
def test_gradient_over_many_rows_of_positive_values(dtype, K, N, rows):
    # Rows repeat with a period, so that the sum in 64 bits is short.
    gen = torch.Generator().manual_seed(K)
    period = 4096
    x = ((torch.rand(period, K, generator=gen) + 1) * 2.0 ** -4).to(dtype).cuda()
    dy = ((torch.rand(period, N, generator=gen) + 1) * 2.0 ** -7).to(dtype).cuda()
    index = (torch.arange(rows, device="cuda") % period).to(torch.int32)
    dw = tmm.gemm_grouped_wgrad(x, dy[index.long()], offsets_of([0, rows]).cuda(), rows=index)
    tmm.check_device()
    whole, rest = divmod(rows, period)
    want = whole * (x.double().T @ dy.double()) + x[:rest].double().T @ dy[:rest].double()
    assert not dw[0].any()
    sums_within(dw[1], want, rows)


@pytest.mark.parametrize("dtype", TYPES[:2], ids=str)
@pytest.mark.parametrize("rows,N", [(300, 256), (5, 72)])
def test_long_rows_of_positive_values(dtype, rows, N):
    gen = torch.Generator().manual_seed(rows)
    K = 2 ** 19 + 8
    x = ((torch.rand(rows, K, generator=gen) + 1) * 2.0 ** -4).to(dtype).cuda()
    w = ((torch.rand(1, N, K, generator=gen) + 1) * 2.0 ** -7).to(dtype).cuda()
    y = tmm.gemm_grouped(x, w.transpose(1, 2), offsets_of([rows]).cuda())
    tmm.check_device()
    sums_within(y, x.double() @ w[0].double().T, K)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("sizes,K,N", [([300, 0, 257], 9001, 264), ([3, 1], 9001, 264),
                                       ([40], 16384, 72), ([513], 25000, 140)])
def test_integers_of_long_sums_are_exact(dtype, sizes, K, N):
    gen = torch.Generator().manual_seed(K + N)
    R = sum(sizes)
    x, w, off = ints(gen, R, K), ints(gen, len(sizes), K, N), offsets_of(sizes)
    y = tmm.gemm_grouped(x.to(dtype).cuda(), w.to(dtype).cuda(), off.cuda())
    tmm.check_device()
    assert torch.equal(y.cpu(), ref.grouped(x, w, off).to(dtype))


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("sizes,K,N", [([9001, 100, 0, 16385], 130, 264), ([8200, 8192, 24577], 70, 72)])
def test_integers_of_many_rows_are_exact(dtype, sizes, K, N):
    gen = torch.Generator().manual_seed(K + N)
    R = sum(sizes)
    x, dy, off = ints(gen, R, K), ints(gen, R, N), offsets_of(sizes)
    dw = tmm.gemm_grouped_wgrad(x.to(dtype).cuda(), dy.to(dtype).cuda(), off.cuda())
    tmm.check_device()
    assert torch.equal(dw.cpu(), ref.wgrad(x, dy, off).to(dtype))


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("K,r", [(8192, 24), (8200, 40), (17000, 70)])
@pytest.mark.parametrize("sizes,first,T", [([9] * 60, 0, 600), ([255, 0, 257], 33, 573),
                                           ([1, 2], 0, 5)])
def test_adapters_beside_long_sums_are_exact(dtype, sizes, first, T, K, r):
    gen = torch.Generator().manual_seed(K + r + T)
    L, N = len(sizes), 300
    x, w = ints(gen, T, K), ints(gen, K, N)
    a, b = ints(gen, L, K, r), ints(gen, L, r, N)
    a *= torch.rand(L, K, 1, generator=gen) < 0.02
    off, scale = offsets_of(sizes, first), torch.tensor([2.0 ** (i % 3 - 1) for i in range(L)])
    y = tmm.gemm_lora(x.to(dtype).cuda(), w.to(dtype).cuda(), a.to(dtype).cuda(),
                      b.to(dtype).cuda(), scale.cuda(), off.cuda())
    tmm.check_device()
    assert torch.equal(y.cpu(), ref.lora(x, w, a, b, scale, off).to(dtype))


@pytest.mark.parametrize("dtype", [torch.float32], ids=str)
@pytest.mark.parametrize("sizes,K,N", [([300, 257], 9001, 264), ([3, 1], 65536, 264)])
def test_random_long_sums_in_single_precision(dtype, sizes, K, N):
    gen = torch.Generator().manual_seed(K + N)
    x = torch.randn(sum(sizes), K, generator=gen)
    w, off = torch.randn(len(sizes), K, N, generator=gen), offsets_of(sizes)
    y = tmm.gemm_grouped(x.cuda(), w.cuda(), off.cuda())
    tmm.check_device()
    want = ref.grouped(x, w, off)
    ref.assert_within(y, want, ref.grouped(x.abs(), w.abs(), off), K)
    assert (y.double().cpu() - want).norm() <= 1e-6 * want.norm()


def test_single_precision_whose_lower_parts_have_one_sign():
    # x = x0 + x1 with x0 of eight bits and x1 between 0.1 and 0.9 half steps of it, dy likewise:
    # the sums of x1 dy0 and x0 dy1 only grow.  The additions of FP32 registers are rounded to
    # nearest and their errors of either sign; what is left on the mean over all results is the
    # tensor core's: TAKEN_FP32 / 16 additions of 2^-22 of the partial sum for the leading products,
    # and five times as many for the others, of 2^-7 of the size at most.
    gen = torch.Generator().manual_seed(0)
    period, rows, K, N = 4096, 2 ** 20, 64 * 77, 16

    def values(n):
        top = torch.randint(128, 256, (period, n), generator=gen) / 256.0
        return top + (torch.rand(period, n, generator=gen) * 0.8 + 0.1) * 2.0 ** -9
    x, dy = values(K).cuda(), values(N).cuda()
    index = (torch.arange(rows, device="cuda") % period).to(torch.int32)
    dw = tmm.gemm_grouped_wgrad(x, dy[index.long()], offsets_of([rows]).cuda(), rows=index)[0]
    tmm.check_device()
    want = rows // period * (x.double().T @ dy.double())
    mean = ((dw.double() - want) / want).mean().item()
    assert abs(mean) <= TAKEN_FP32 / 16 * 2.0 ** -22 + 5 * TAKEN_FP32 / 16 * 2.0 ** -22 * 2.0 ** -7, mean
