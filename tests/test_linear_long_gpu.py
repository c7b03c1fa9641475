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


@pytest.mark.parametrize("dtype,N", [(torch.float32, 29312), (torch.float32, 136),
                                     (torch.bfloat16, 58632)], ids=str)
def test_sums_of_wide_biases_over_many_rows(dtype, N):
    """Errors do not grow with the rows beyond those of runs of 4096: a thread adds 512 terms of
    one, eight threads' are added, a thread adds an eighth of the 16 runs' sums, and eight are added: 530
    additions that a term passes through at most, half a step of the sum so far each.  The values
    lose all but half a step of sums between 2048 and 4096 and more, always downwards."""
    rows = 65536
    value = (1 + 2.0 ** -12 - 2.0 ** -23) if dtype is torch.float32 else 1 + 2.0 ** -7
    dy = torch.full((rows, N), value, dtype=dtype, device="cuda")
    if dtype is torch.bfloat16:      # dz = dy s(z): the products are FP32 values of no few bits
        pre = torch.full((1, 1), 0.6875, dtype=dtype, device="cuda").expand(rows, N).contiguous()
        got = tmm.gemm_bias_act_grad(dy, None, None, pre=pre, act="silu", dx=False, dw=False,
                                     dbias=True).dbias
        one = tmm.gemm_bias_act_grad(dy[:1], None, None, pre=pre[:1], act="silu", dx=False, dw=False,
                                     dbias=True).dbias
        want = float(one[0]) * rows
    else:
        got = tmm.gemm_bias_act_grad(dy, None, None, dx=False, dw=False, dbias=True).dbias
        want = float(dy[0, 0]) * rows
    off = float((got.double() - want).abs().max()) / want
    assert off <= 530 * 2.0 ** -24, off * 2 ** 24
