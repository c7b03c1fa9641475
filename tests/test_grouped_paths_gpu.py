"""Paths of the grouped operators that only larger sizes take, and rows that nothing names."""
import pytest

torch = pytest.importorskip("torch")

import grouped_ref as ref  # noqa: E402
import tiled_matrix_multiply_gb300 as tmm  # noqa: E402

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]


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


def put(t, dtype, trans):
    return t.transpose(-1, -2).contiguous().to(dtype).cuda().transpose(-1, -2) if trans \
        else t.to(dtype).cuda()


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("sizes,T,r", [([1500, 1200, 0, 1800, 1300, 2000], 8192, 256),
                                       ([2000, 0, 1900], 4000, 1024), ([700, 650], 1400, 1000)])
def test_adapters_of_high_rank(dtype, trans, sizes, T, r):
    # The product with a is large enough for pairs of blocks.
    gen = torch.Generator().manual_seed(r)
    K, N, L = 96, 264, len(sizes)
    x, w = ints(gen, T, K), ints(gen, K, N)
    a, b = ints(gen, L, K, r), ints(gen, L, r, N)
    a *= torch.rand(L, K, 1, generator=gen) < 0.2
    off, scale = offsets_of(sizes, 3), torch.tensor([2.0 ** (i % 3 - 1) for i in range(L)])
    order = torch.randperm(T, generator=gen).to(torch.int32)
    y = tmm.gemm_lora(put(x, dtype, False), put(w, dtype, trans), put(a, dtype, trans),
                      put(b, dtype, trans), scale.cuda(), off.cuda(), rows=order.cuda())
    tmm.check_device()
    assert torch.equal(y.cpu(), ref.lora(x, w, a, b, scale, off, order).to(dtype))


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("by_index", [False, True])
@pytest.mark.parametrize("sizes,K,N", [([5000], 200, 16), ([2100, 0, 3001], 96, 100),
                                       ([4097, 2048], 130, 128)])
def test_gradient_of_few_columns_over_many_rows(dtype, by_index, sizes, K, N):
    # Blocks of a cluster share a group's sum.
    gen = torch.Generator().manual_seed(K + N)
    R, X = sum(sizes), 300
    x, dy = ints(gen, X if by_index else R, K), ints(gen, R, N)
    rows = torch.randint(-1, X + 2, (R,), generator=gen).to(torch.int32) if by_index else None
    off = offsets_of(sizes)
    dw = tmm.gemm_grouped_wgrad(x.to(dtype).cuda(), dy.to(dtype).cuda(), off.cuda(),
                                rows=None if rows is None else rows.cuda())
    tmm.check_device()
    assert torch.equal(dw.cpu(), ref.wgrad(x, dy, off, rows).to(dtype))


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("T,K", [(20, 72), (20, 4000), (300, 72), (600, 72)])
@pytest.mark.parametrize("N,pad", [(136, 0), (136, 8), (131, 0), (136, 3)])
def test_rows_that_the_order_does_not_name_are_not_written(dtype, T, K, N, pad):
    gen = torch.Generator().manual_seed(T + K + N + pad)
    L, r = 3, 8
    x, w = ints(gen, T, K), ints(gen, K, N)
    a, b = ints(gen, L, K, r), ints(gen, L, r, N)
    a *= torch.rand(L, K, 1, generator=gen) < 20.0 / K
    sizes = [T // 4, 0, T // 2]
    off, scale = offsets_of(sizes, 1), torch.ones(L)
    order = torch.randperm(T, generator=gen).to(torch.int32)
    lost = torch.rand(T, generator=gen) < 0.3
    lost[:2] = True
    unnamed = order[lost].long()
    named = order.clone()
    named[lost] = torch.where(torch.arange(int(lost.sum())) % 2 == 0, -1, T).to(torch.int32)
    buf = torch.full((T, N + pad), float("nan"), dtype=dtype, device="cuda")
    y = buf[:, :N]
    tmm.gemm_lora(x.to(dtype).cuda(), w.to(dtype).cuda(), a.to(dtype).cuda(), b.to(dtype).cuda(),
                  scale.cuda(), off.cuda(), rows=named.cuda(), y=y)
    tmm.check_device()
    want = ref.lora(x, w, a, b, scale, off, order)       # rows of the places that keep theirs
    want[unnamed] = float("nan")
    got = buf.cpu()
    assert torch.isnan(got[unnamed]).all() and torch.isnan(got[:, N:]).all()
    keep = torch.ones(T, dtype=torch.bool)
    keep[unnamed] = False
    assert torch.equal(got[keep][:, :N], want[keep].to(dtype))
