"""A call of the grouped operators whose waits run out ends soon, however many tiles it has."""
import time

import pytest

torch = pytest.importorskip("torch")

import tiled_matrix_multiply_gb300 as tmm  # noqa: E402
from tiled_matrix_multiply_gb300 import _abi  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tiled_matrix_multiply_gb300 import build
    build.build()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
def test_waits_run_out_once_a_call(dtype):
    # Adapters of few rows meet at every tile: one block has 24 of them.  Its roles wait one after
    # another, each for what the one before did not do: eight limits hold them all.
    lib, limit = _abi.load(), 0.1
    T, K, N, r = 64, 64, 152 * 128 * 24, 8
    x, w = torch.ones(T, K, dtype=dtype, device="cuda"), torch.ones(K, N, dtype=dtype, device="cuda")
    a = torch.zeros(1, K, r, dtype=dtype, device="cuda")
    b = torch.zeros(1, r, N, dtype=dtype, device="cuda")
    args = (x, w, a, b, torch.ones(1, device="cuda"),
            torch.tensor([0, T], dtype=torch.int32, device="cuda"))
    want = tmm.gemm_lora(*args)
    tmm.check_device()
    lib.tmm_testing_set_wait_hooks(0, int(limit * 1e9))
    try:
        start = time.perf_counter()
        tmm.gemm_lora(*args)
        with pytest.raises(tmm.TmmError) as e:
            tmm.check_device()
        took = time.perf_counter() - start
        assert e.value.status == _abi.TMM_ERR_DEVICE_TIMEOUT
    finally:
        lib.tmm_testing_set_wait_hooks(-1, 0)
    assert took <= 8 * limit, took
    assert torch.equal(tmm.gemm_lora(*args), want)
    tmm.check_device()
