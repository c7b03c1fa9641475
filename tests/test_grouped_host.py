"""The grouped operators on the host: refusals before any CUDA call, workspace sizes, and the
64-bit definitions that the GPU tests compare with (CPU only; no compute call is made)."""
import itertools

import pytest

torch = pytest.importorskip("torch")

import grouped_ref as ref  # noqa: E402
from tiled_matrix_multiply_gb300 import _abi, build  # noqa: E402

FAKE = 0x7F0000001000          # never dereferenced: every case fails validation first
FAR = [FAKE + (i << 40) for i in range(12)]


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _abi.load()


def grouped_args(**change):
    a = dict(dtype=_abi.TMM_BF16, transw=0, groups=4, rows=16, N=64, K=128, x=FAR[0], x_rows=16,
             ldx=128, offsets=FAR[1], row_index=0, w=FAR[2], ldw=64, stride_w=128 * 64, y=FAR[3],
             ldy=64, ws=0, ws_bytes=0, stream=None)
    a.update(change)
    return list(a.values())


@pytest.mark.parametrize("change,status", [
    (dict(dtype=3), _abi.TMM_ERR_INVALID_ARG),
    (dict(dtype=-1), _abi.TMM_ERR_INVALID_ARG),
    (dict(transw=2), _abi.TMM_ERR_INVALID_ARG),
    (dict(groups=0), _abi.TMM_ERR_INVALID_ARG),
    (dict(groups=513), _abi.TMM_ERR_INVALID_ARG),
    (dict(rows=-1), _abi.TMM_ERR_INVALID_ARG),
    (dict(rows=1 << 29, x_rows=1 << 29), _abi.TMM_ERR_INVALID_ARG),
    (dict(N=-1), _abi.TMM_ERR_INVALID_ARG),
    (dict(K=1 << 30), _abi.TMM_ERR_INVALID_ARG),
    (dict(x_rows=15), _abi.TMM_ERR_INVALID_ARG),                  # fewer rows than are read
    (dict(x_rows=-1, row_index=FAR[4]), _abi.TMM_ERR_INVALID_ARG),
    (dict(ldx=127), _abi.TMM_ERR_INVALID_ARG),
    (dict(ldw=63), _abi.TMM_ERR_INVALID_ARG),
    (dict(transw=1, ldw=127), _abi.TMM_ERR_INVALID_ARG),
    (dict(ldy=63), _abi.TMM_ERR_INVALID_ARG),
    (dict(stride_w=-1), _abi.TMM_ERR_INVALID_ARG),
    (dict(stride_w=1 << 60, ldw=64), _abi.TMM_ERR_INVALID_ARG),   # extent beyond 64 bits
    (dict(x=0), _abi.TMM_ERR_INVALID_ARG),
    (dict(w=0), _abi.TMM_ERR_INVALID_ARG),
    (dict(y=0), _abi.TMM_ERR_INVALID_ARG),
    (dict(offsets=0), _abi.TMM_ERR_INVALID_ARG),
    (dict(x=FAR[0] + 1), _abi.TMM_ERR_INVALID_ARG),
    (dict(offsets=FAR[1] + 2), _abi.TMM_ERR_INVALID_ARG),
    (dict(row_index=FAR[4] + 1), _abi.TMM_ERR_INVALID_ARG),
    (dict(x=FAR[0] + 2), _abi.TMM_ERR_INVALID_ARG),               # restaged: workspace missing
    (dict(x=FAR[0] + 2, ws=FAR[5], ws_bytes=100), _abi.TMM_ERR_INVALID_ARG),
    (dict(x=FAR[0] + 2, ws=FAR[5] + 128, ws_bytes=1 << 20), _abi.TMM_ERR_INVALID_ARG),
    (dict(y=FAR[0] + 64), _abi.TMM_ERR_ALIAS),
    (dict(y=FAR[2] + 4096), _abi.TMM_ERR_ALIAS),
    (dict(y=FAR[1] - 1024), _abi.TMM_ERR_ALIAS),                  # over the offsets
    (dict(x=FAR[0] + 2, ws=FAR[2], ws_bytes=1 << 20), _abi.TMM_ERR_ALIAS),
    (dict(x=FAR[0] + 2, ws=FAR[3], ws_bytes=1 << 20), _abi.TMM_ERR_ALIAS),
])
def test_grouped_refusals(lib, change, status):
    assert lib.gemm_grouped(*grouped_args(**change)) == status
    assert lib.tmm_last_error_string().decode()


@pytest.mark.parametrize("change", [dict(rows=0), dict(N=0, ldw=1, ldy=1, stride_w=128)])
def test_grouped_nothing_to_do_needs_no_device(lib, change):
    assert lib.gemm_grouped(*grouped_args(**change)) == _abi.TMM_OK


def wgrad_args(**change):
    a = dict(dtype=_abi.TMM_F16, groups=4, rows=16, N=64, K=128, x=FAR[0], x_rows=16, ldx=128,
             offsets=FAR[1], row_index=0, dy=FAR[2], lddy=64, dw=FAR[3], lddw=64,
             stride_dw=128 * 64, ws=0, ws_bytes=0, stream=None)
    a.update(change)
    return list(a.values())


@pytest.mark.parametrize("change,status", [
    (dict(dtype=7), _abi.TMM_ERR_INVALID_ARG),
    (dict(groups=-1), _abi.TMM_ERR_INVALID_ARG),
    (dict(x_rows=3), _abi.TMM_ERR_INVALID_ARG),
    (dict(lddy=10), _abi.TMM_ERR_INVALID_ARG),
    (dict(lddw=10), _abi.TMM_ERR_INVALID_ARG),
    (dict(stride_dw=128 * 64 - 1), _abi.TMM_ERR_INVALID_ARG),     # matrices would overlap
    (dict(stride_dw=0), _abi.TMM_ERR_INVALID_ARG),
    (dict(dy=0), _abi.TMM_ERR_INVALID_ARG),
    (dict(dw=0), _abi.TMM_ERR_INVALID_ARG),
    (dict(dy=FAR[2] + 2), _abi.TMM_ERR_INVALID_ARG),              # restaged: workspace missing
    (dict(dw=FAR[0]), _abi.TMM_ERR_ALIAS),
    (dict(dw=FAR[2] + 16), _abi.TMM_ERR_ALIAS),
])
def test_wgrad_refusals(lib, change, status):
    assert lib.gemm_grouped_wgrad(*wgrad_args(**change)) == status
    assert lib.tmm_last_error_string().decode()


def lora_args(**change):
    a = dict(dtype=_abi.TMM_BF16, transw=0, transa=0, transb=0, groups=4, rows=16, N=64, K=128,
             rank=8, x=FAR[0], ldx=128, offsets=FAR[1], row_index=0, w=FAR[2], ldw=64, a=FAR[3],
             lda=8, stride_a=1024, b=FAR[4], ldb=64, stride_b=512, scale=FAR[5], y=FAR[6], ldy=64,
             ws=FAR[7], ws_bytes=1 << 20, stream=None)
    a.update(change)
    return list(a.values())


@pytest.mark.parametrize("change,status", [
    (dict(transa=2), _abi.TMM_ERR_INVALID_ARG),
    (dict(transb=-1), _abi.TMM_ERR_INVALID_ARG),
    (dict(rank=0), _abi.TMM_ERR_INVALID_ARG),
    (dict(rank=1025, lda=1025), _abi.TMM_ERR_INVALID_ARG),
    (dict(lda=7), _abi.TMM_ERR_INVALID_ARG),
    (dict(ldb=63), _abi.TMM_ERR_INVALID_ARG),
    (dict(transb=1, ldb=7), _abi.TMM_ERR_INVALID_ARG),
    (dict(scale=0), _abi.TMM_ERR_INVALID_ARG),
    (dict(scale=FAR[5] + 2), _abi.TMM_ERR_INVALID_ARG),
    (dict(a=0), _abi.TMM_ERR_INVALID_ARG),
    (dict(ws=0, ws_bytes=0), _abi.TMM_ERR_INVALID_ARG),
    (dict(ws_bytes=16), _abi.TMM_ERR_INVALID_ARG),
    (dict(y=FAR[3] + 64), _abi.TMM_ERR_ALIAS),
    (dict(y=FAR[4]), _abi.TMM_ERR_ALIAS),
    (dict(y=FAR[5] - 64), _abi.TMM_ERR_ALIAS),
    (dict(ws=FAR[4]), _abi.TMM_ERR_ALIAS),
    (dict(ws=FAR[6]), _abi.TMM_ERR_ALIAS),
])
def test_lora_refusals(lib, change, status):
    assert lib.gemm_lora(*lora_args(**change)) == status
    assert lib.tmm_last_error_string().decode()


def rows_args(**change):
    a = dict(tokens=100, fan=2, groups=8, index=FAR[0], bits=32, offsets=FAR[1], order=FAR[2],
             rows=FAR[3], position=FAR[4], ws=0, ws_bytes=0, stream=None)
    a.update(change)
    return list(a.values())


@pytest.mark.parametrize("change,status", [
    (dict(tokens=-1), _abi.TMM_ERR_INVALID_ARG),
    (dict(fan=0), _abi.TMM_ERR_INVALID_ARG),
    (dict(tokens=1 << 30, fan=2), _abi.TMM_ERR_INVALID_ARG),
    (dict(groups=0), _abi.TMM_ERR_INVALID_ARG),
    (dict(groups=513), _abi.TMM_ERR_INVALID_ARG),
    (dict(bits=16), _abi.TMM_ERR_INVALID_ARG),
    (dict(index=0), _abi.TMM_ERR_INVALID_ARG),
    (dict(bits=64, index=FAR[0] + 4), _abi.TMM_ERR_INVALID_ARG),
    (dict(offsets=0), _abi.TMM_ERR_INVALID_ARG),
    (dict(order=0), _abi.TMM_ERR_INVALID_ARG),
    (dict(position=0), _abi.TMM_ERR_INVALID_ARG),
    (dict(tokens=100000), _abi.TMM_ERR_INVALID_ARG),              # workspace missing
    (dict(order=FAR[0] + 8), _abi.TMM_ERR_ALIAS),
    (dict(position=FAR[2]), _abi.TMM_ERR_ALIAS),
    (dict(rows=FAR[1]), _abi.TMM_ERR_ALIAS),
])
def test_group_rows_refusals(lib, change, status):
    assert lib.group_rows(*rows_args(**change)) == status
    assert lib.tmm_last_error_string().decode()


def test_workspace_sizes(lib):
    def grouped(dtype, rows, x=FAR[0], ldx=128, index=0, K=128, N=256, groups=4):
        return lib.gemm_grouped_workspace_size(dtype, 0, groups, rows, N, K, x, rows, ldx, index,
                                               FAR[2], N, K * N)
    # 16-bit operands on 16-byte boundaries are read in place, few rows by their number too;
    # FP32 with few rows is split on the way.
    assert grouped(_abi.TMM_BF16, 16) == grouped(_abi.TMM_BF16, 16, index=FAR[3]) == 0
    assert grouped(_abi.TMM_F32, 16) == 0
    # Off a boundary: a copy whose rows are multiples of eight values, in 256-byte sections.
    assert grouped(_abi.TMM_BF16, 16, x=FAR[0] + 2) == 16 * 128 * 2
    assert grouped(_abi.TMM_F16, 5, x=FAR[0] + 2, ldx=129) == 5 * 128 * 2
    # Rows by number are gathered where pairs of blocks have work for all, not with fewer tiles;
    # FP32 has three planes of x and w there.
    assert grouped(_abi.TMM_BF16, 4096, index=FAR[3]) == 0
    assert grouped(_abi.TMM_BF16, 65536, index=FAR[3], groups=1) == 65536 * 128 * 2
    assert grouped(_abi.TMM_F32, 65536, groups=1) == 65536 * 128 * 6 + 128 * 256 * 6
    # Sizes that a call would refuse need nothing; counts past size_t say so.
    assert grouped(9, 16) == 0
    assert lib.gemm_grouped_workspace_size(_abi.TMM_F32, 0, 0, 16, 256, 128, FAR[0], 16, 128, 0,
                                           FAR[2], 256, 0) == 0
    big = (1 << 29) - 1
    assert lib.gemm_grouped_workspace_size(_abi.TMM_F32, 0, 512, big, big, big, FAR[0], big, big, 0,
                                           FAR[2], big, big * big) == 2 ** 64 - 1
    assert lib.group_rows_workspace_size(2048, 1, 8) == 0
    assert lib.group_rows_workspace_size(2049, 1, 8) == 256 * 9 * 4


def test_python_refusals_on_the_cpu():
    import tiled_matrix_multiply_gb300 as tmm
    f, i = torch.zeros, torch.int32
    with pytest.raises(ValueError):
        tmm.gemm_grouped(f(4, 8), f(2, 8, 8), f(3, dtype=i))           # host tensors
    with pytest.raises(TypeError):
        tmm.gemm_grouped(f(4, 8, dtype=torch.float64), f(2, 8, 8), f(3, dtype=i))
    with pytest.raises(TypeError):
        tmm.gemm_grouped(None, f(2, 8, 8), f(3, dtype=i))
    with pytest.raises(TypeError):
        tmm.group_rows(f(4, 2), 3)
    with pytest.raises(ValueError):
        tmm.group_rows(f(4, 2, dtype=i), 3)
    with pytest.raises(ValueError):
        tmm.gemm_grouped_wgrad(f(4, 8), f(4, 8), f(3, dtype=i))
    with pytest.raises(ValueError):
        tmm.gemm_lora(f(4, 8), f(8, 8), f(2, 8, 2), f(2, 2, 8), f(2), f(3, dtype=i))


def test_definitions_by_brute_force():
    gen = torch.Generator().manual_seed(0)
    off, R, K, N, G = [2, 1, 4, 9], 6, 3, 2, 3
    x = torch.randint(-3, 4, (5, K), generator=gen).double()
    w = torch.randint(-3, 4, (G, K, N), generator=gen).double()
    rows = torch.tensor([0, 4, 9, -1, 2, 2], dtype=torch.int32)
    b = [2, 2, 4, 6]                # clamped to [0, R], never stepping back
    assert ref.bounds(off, R) == b
    y = torch.zeros(R, N).double()
    dy = torch.randint(-3, 4, (R, N), generator=gen).double()
    dw = torch.zeros(G, K, N).double()
    for g, p in itertools.product(range(G), range(R)):
        if b[g] <= p < b[g + 1] and 0 <= int(rows[p]) < 5:
            for k, n in itertools.product(range(K), range(N)):
                y[p, n] += x[rows[p], k] * w[g, k, n]
                dw[g, k, n] += x[rows[p], k] * dy[p, n]
    assert torch.equal(ref.grouped(x, w, off, rows), y)
    assert torch.equal(ref.wgrad(x, dy, off, rows), dw)
