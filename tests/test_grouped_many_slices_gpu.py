"""Long sums of tiles in which some of the copying warps have nothing to copy."""
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


def ints(gen, *shape):
    return torch.randint(-1, 2, shape, generator=gen).double()


def offsets_of(sizes):
    return torch.tensor([0] + sizes).cumsum(0).to(torch.int32)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("by_index", [False, True])
@pytest.mark.parametrize("sizes,K,N", [([1, 0, 4, 2], 6000, 2500), ([257, 513, 1, 300], 4000, 700),
                                       ([1], 8000, 40)])
def test_products(dtype, by_index, sizes, K, N):
    # Groups of one row (one copy of four rows by number, for three warps), and tiles of pairs whose
    # second half holds no row.
    gen = torch.Generator().manual_seed(K + N)
    R, X = sum(sizes), 50
    x, w = ints(gen, X if by_index else R, K), ints(gen, len(sizes), K, N)
    rows = torch.randint(-1, X + 2, (R,), generator=gen).to(torch.int32) if by_index else None
    off = offsets_of(sizes)
    want = ref.grouped(x, w, off, rows).to(dtype).cuda()
    args = (x.to(dtype).cuda(), w.to(dtype).cuda(), off.cuda())
    index = None if rows is None else rows.cuda()
    same = torch.ones((), dtype=torch.bool, device="cuda")
    for _ in range(50):
        same &= (tmm.gemm_grouped(*args, rows=index) == want).all()
    tmm.check_device()
    assert bool(same)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("sizes,N", [([3000, 1, 0, 2049], 40), ([700, 64, 3], 100)])
def test_gradients(dtype, sizes, N):
    gen = torch.Generator().manual_seed(N)
    R, X, K = sum(sizes), 60, 70
    x, dy = ints(gen, X, K), ints(gen, R, N)
    rows = torch.randint(-1, X + 2, (R,), generator=gen).to(torch.int32)
    off = offsets_of(sizes)
    want = ref.wgrad(x, dy, off, rows).to(dtype).cuda()
    args = (x.to(dtype).cuda(), dy.to(dtype).cuda(), off.cuda())
    same = torch.ones((), dtype=torch.bool, device="cuda")
    for _ in range(50):
        same &= (tmm.gemm_grouped_wgrad(*args, rows=rows.cuda()) == want).all()
    tmm.check_device()
    assert bool(same)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("sizes,T", [([300, 233, 0], 545), ([1024, 1], 1056)])
def test_adapters(dtype, sizes, T):
    gen = torch.Generator().manual_seed(T)
    K, N, L, r = 4000, 700, len(sizes), 8
    x, w, a, b = ints(gen, T, K), ints(gen, K, N), ints(gen, L, K, r), ints(gen, L, r, N)
    a *= torch.rand(L, K, 1, generator=gen) < 0.02
    off, scale = offsets_of(sizes), torch.ones(L)
    want = ref.lora(x, w, a, b, scale, off).to(dtype).cuda()
    args = [t.to(dtype).cuda() for t in (x, w, a, b)] + [scale.cuda(), off.cuda()]
    same = torch.ones((), dtype=torch.bool, device="cuda")
    for _ in range(50):
        same &= (tmm.gemm_lora(*args) == want).all()
    tmm.check_device()
    assert bool(same)
