"""A linear layer whose waits run out ends soon, says so, and leaves the next call whole."""
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


# A shared sum, single blocks with several tiles each, pairs with several tiles each.
@pytest.mark.parametrize("M,K,N", [(16, 2048, 1024), (16, 64, 128 * 152 * 5), (4096, 512, 4096)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=str)
def test_waits_run_out_once_a_call(dtype, M, K, N):
    lib, limit = _abi.load(), 0.1
    if dtype is torch.float32:
        M = max(M, 17)      # of fewer rows the FP32 units' kernel waits for nothing
    x, w = torch.ones(M, K, dtype=dtype, device="cuda"), torch.ones(K, N, dtype=dtype, device="cuda")
    want = tmm.gemm_bias_act(x, w)
    tmm.check_device()
    lib.tmm_testing_set_wait_hooks(0, int(limit * 1e9))
    try:
        start = time.perf_counter()
        tmm.gemm_bias_act(x, w)
        with pytest.raises(tmm.TmmError) as e:
            tmm.check_device()
        took = time.perf_counter() - start
        assert e.value.status == _abi.TMM_ERR_DEVICE_TIMEOUT
    finally:
        lib.tmm_testing_set_wait_hooks(-1, 0)
    assert took <= 8 * limit, took
    assert torch.equal(tmm.gemm_bias_act(x, w), want)
    tmm.check_device()
