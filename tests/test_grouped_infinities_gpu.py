"""Infinite entries: results are infinite, or NaN, where the definition's are."""
import pytest

torch = pytest.importorskip("torch")

import grouped_ref as ref  # noqa: E402
import tiled_matrix_multiply_gb300 as tmm  # noqa: E402

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tiled_matrix_multiply_gb300 import build
    build.build()


def ints(gen, *shape):
    return torch.randint(-2, 3, shape, generator=gen).double()


def plant(gen, t, share):
    t[torch.rand(t.shape, generator=gen) < share] = INF
    t[torch.rand(t.shape, generator=gen) < share] = -INF
    return t


def same(got, want):
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got, nan=7.0), torch.nan_to_num(want, nan=7.0))


SIZES = [([3, 0, 2], 700, 72), ([3, 2], 200, 136), ([60, 200], 300, 264), ([600, 513], 200, 264)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=str)
@pytest.mark.parametrize("sizes,K,N", SIZES)
@pytest.mark.parametrize("share", [0.0005, 0.02])
def test_infinite_entries(sizes, K, N, share, dtype):
    gen = torch.Generator().manual_seed(K + N)
    R = sum(sizes)
    off = torch.tensor([0] + sizes).cumsum(0).to(torch.int32)
    x, w, dy = (plant(gen, ints(gen, *s), share) for s in ((R, K), (len(sizes), K, N), (R, N)))
    y = tmm.gemm_grouped(x.to(dtype).cuda(), w.to(dtype).cuda(), off.cuda()).cpu()
    same(y, ref.grouped(x, w, off).to(dtype))
    dw = tmm.gemm_grouped_wgrad(x.to(dtype).cuda(), dy.to(dtype).cuda(), off.cuda()).cpu()
    same(dw, ref.wgrad(x, dy, off).to(dtype))
    tmm.check_device()


@pytest.mark.parametrize("T", [20, 300, 900])
@pytest.mark.parametrize("share", [0.0005, 0.01])
def test_infinite_entries_of_adapters(T, share):
    gen = torch.Generator().manual_seed(T)
    K, N, L, r = 200, 264, 3, 12
    off, scale = torch.tensor([0, T // 3, T // 3, T - 2], dtype=torch.int32), torch.ones(L)
    x, w, a, b = (plant(gen, ints(gen, *s), share)
                  for s in ((T, K), (K, N), (L, K, r), (L, r, N)))
    y = tmm.gemm_lora(x.float().cuda(), w.float().cuda(), a.float().cuda(), b.float().cuda(),
                      scale.cuda(), off.cuda()).cpu()
    tmm.check_device()
    same(y, ref.lora(x, w, a, b, scale, off).float())
