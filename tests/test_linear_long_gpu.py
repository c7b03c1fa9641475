"""Linear layers of long calls and long sums."""
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


@pytest.mark.parametrize("dtype,size", [(torch.bfloat16, 16384), (torch.float32, 8192)], ids=str)
def test_a_call_may_take_longer_than_a_wait(dtype, size):
    """The limit is each wait's, of some 0.1 ms at most here; the calls take 4 ms and more."""
    x = torch.ones(size, size, dtype=dtype, device="cuda")
    lib = _abi.load()
    tmm.gemm_bias_act(x, x)
    tmm.check_device()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    lib.tmm_testing_set_wait_hooks(-1, 1500 * 1000)
    try:
        start.record()
        y = tmm.gemm_bias_act(x, x)
        end.record()
        tmm.check_device()
    finally:
        lib.tmm_testing_set_wait_hooks(-1, 0)
    assert start.elapsed_time(end) > 2.5
    assert bool((y == size).all())
