"""What an adapter's inner product u = scale[g] (x a[g]) keeps on its way to b[g], on the GPU.

u has FP32's range whatever the type of the matrices and the number of rows, and at least 17 bits
(bf16; 24 in fp16 and fp32) of any value: values beyond the type's range, values far below its
steps, and the bits that it rounds off all reach the product with b.
"""
import pytest

torch = pytest.importorskip("torch")

import grouped_ref as ref  # noqa: E402
import tiled_matrix_multiply_gb300 as tmm  # noqa: E402

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]
HALVES = TYPES[:2]


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tiled_matrix_multiply_gb300 import build
    build.build()


def put(t, dtype, trans=False):
    return t.transpose(-1, -2).contiguous().to(dtype).cuda().transpose(-1, -2) if trans \
        else t.to(dtype).cuda()


def between(gen, lo, hi, *shape):
    return torch.randint(lo, hi + 1, shape, generator=gen).double()


def lora(x, w, a, b, scale, off, dtype, trans=False):
    y = tmm.gemm_lora(put(x, dtype), put(w, dtype), put(a, dtype), put(b, dtype, trans),
                      scale.cuda(), torch.tensor(off, dtype=torch.int32).cuda())
    tmm.check_device()
    return y.cpu()


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("r", [8, 40])
@pytest.mark.parametrize("T", [20, 600])
def test_u_beyond_the_range_of_the_type(dtype, trans, r, T):
    # u between 57600 and 230400 (fp16 ends at 65504), b multiples of 2^-9 or zero: every partial
    # sum is a multiple of 2^-9 below 2^15, so FP32 sums are exact and only the result is rounded
    # (bf16: and u, which has 18 bits, to 17).
    gen = torch.Generator().manual_seed(T + r)
    K, N, L = 64, 140, 3
    x, a = between(gen, 30, 60, T, K), between(gen, 30, 60, L, K, r)
    w = between(gen, -1, 1, K, N)
    b = between(gen, -1, 1, L, r, N) * 2.0 ** -9
    b *= torch.rand(L, r, N, generator=gen) < 0.3
    b[1] = 0.0                                   # an adapter as it is initialised
    off, scale = [2, T // 4, T // 2, T - 3], torch.ones(L)
    want = ref.lora(x, w, a, b, scale, off)
    assert float(want.abs().max()) < 2 ** 15
    y = lora(x, w, a, b, scale, off, dtype, trans)
    if dtype == torch.bfloat16:
        size = ref.lora(x, torch.zeros_like(w), a, b.abs(), scale, off)
        ref.assert_within(y, want, torch.zeros_like(want), 0, extra=2.0 ** -17 * size)
    else:
        assert torch.equal(y, want.to(dtype))


@pytest.mark.parametrize("dtype", HALVES, ids=str)
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("r", [16, 40, 100])
@pytest.mark.parametrize("T", [20, 600])
def test_all_bits_of_u_reach_the_result(dtype, trans, r, T):
    # w = e - a b, so y = x e: whole numbers up to 255 K, while x a has up to 17 bits (bf16: 16) and
    # x w and u b are of the size of 2^21 each.  Sums of whole numbers below 2^24: exact.
    gen = torch.Generator().manual_seed(T + r)
    K, N, L = 400, 136, 2
    top = 100 if dtype == torch.bfloat16 else 255
    x, a1 = between(gen, 0, top, T, K), between(gen, 1, 4, K, r)
    b1 = between(gen, -1, 1, r, N) * (torch.rand(r, N, generator=gen) < 24 / r)
    e = between(gen, -1, 1, K, N)
    w = e - a1 @ b1
    assert float(w.abs().max()) <= 256
    assert 2 ** 15 < float((x @ a1).max()) < 2 ** 16 or (top == 255 and float((x @ a1).max()) > 2 ** 16)
    assert float((x @ w.abs() + (x @ a1) @ b1.abs()).max()) < 2 ** 24
    a, b = torch.stack([a1] * L), torch.stack([b1] * L)
    y = lora(x, w, a, b, torch.ones(L), [0, T // 3, T], dtype, trans)
    assert torch.equal(y, (x @ e).to(dtype))


@pytest.mark.parametrize("dtype", HALVES, ids=str)
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("size", [2.0 ** -24, 2.0 ** -20, 2.0 ** -12])
@pytest.mark.parametrize("T", [20, 600])
def test_small_u_keeps_its_bits(dtype, trans, size, T):
    # The sums that make u (K terms) and y (its parts' products over the ranks); u itself is off by
    # 2^-17 (bf16), or by 2^-23 and the product of parts that is left out, 2^-23.
    gen = torch.Generator().manual_seed(T)
    K, N, L, r = 128, 136, 2, 24
    x = torch.randn(T, K, generator=gen, dtype=torch.float64).to(dtype)
    a = (torch.randn(L, K, r, generator=gen, dtype=torch.float64) * K ** -0.5).to(dtype)
    b = (torch.randn(L, r, N, generator=gen, dtype=torch.float64) * 2.0 ** 10).to(dtype)
    w = torch.zeros(K, N, dtype=dtype)
    scale = torch.tensor([size, -size])
    off = [0, T // 2, T]
    y = lora(x, w, a, b, scale, off, dtype, trans)
    want = ref.lora(x, w, a, b, scale, off)
    mag = ref.lora(x.abs(), w, a.abs(), b.abs(), scale.abs(), off)
    ref.assert_within(y, want, mag, K + 6 * r,
                      extra=2.0 ** (-17 if dtype == torch.bfloat16 else -22) * mag)


@pytest.mark.parametrize("dtype", HALVES, ids=str)
@pytest.mark.parametrize("T", [20, 600])
def test_infinite_u(dtype, T):
    # Infinite rows of x: u is infinite, and so is u b wherever b is not zero.
    gen = torch.Generator().manual_seed(T)
    K, N, L, r = 64, 136, 2, 24
    x, w = between(gen, 1, 2, T, K), between(gen, 1, 2, K, N)
    a, b = between(gen, 1, 2, L, K, r), between(gen, 1, 2, L, r, N)
    x[3::7, 5] = float("inf")
    y = lora(x, w, a, b, torch.ones(L), [0, T // 2, T], dtype)
    want = ref.lora(x, w, a, b, torch.ones(L), [0, T // 2, T])
    assert torch.equal(y, want.to(dtype))
