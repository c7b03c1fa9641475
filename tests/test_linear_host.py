"""Linear layers on the host: refusals before any CUDA call, workspace sizes, and the 64-bit
definitions (CPU only; no compute call is made)."""
import pytest

torch = pytest.importorskip("torch")

import linear_ref as ref  # noqa: E402
from tiled_matrix_multiply_gb300 import _abi, build  # noqa: E402

FAKE = 0x7F0000001000          # never dereferenced: every case fails validation first
FAR = [FAKE + (i << 40) for i in range(12)]
BAD, ALIAS = _abi.TMM_ERR_INVALID_ARG, _abi.TMM_ERR_ALIAS


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _abi.load()


def args(defaults, change):
    a = dict(defaults)
    assert not set(change) - set(a)
    a.update(change)
    return list(a.values())


LINEAR = dict(dtype=_abi.TMM_BF16, transw=0, act=2, M=16, N=64, K=128, x=FAR[0], ldx=128, w=FAR[1],
              ldw=64, bias=FAR[2], bias_f32=1, residual=FAR[3], ldr=64, y=FAR[4], ldy=64,
              pre=FAR[5], ldpre=64, ws=0, ws_bytes=0, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=3), BAD), (dict(transw=2), BAD), (dict(act=-1), BAD), (dict(act=5), BAD),
    (dict(M=-1), BAD), (dict(N=1 << 29, ldw=1 << 29, ldy=1 << 29, ldr=1 << 29, ldpre=1 << 29), BAD),
    (dict(K=-2), BAD), (dict(ldx=127), BAD), (dict(ldw=63), BAD), (dict(transw=1, ldw=64), BAD),
    (dict(ldr=63), BAD), (dict(ldy=63), BAD), (dict(ldpre=63), BAD), (dict(ldx=1 << 60), BAD),
    (dict(x=0), BAD), (dict(w=0), BAD), (dict(y=0), BAD), (dict(x=FAR[0] + 1), BAD),
    (dict(bias=FAR[2] + 2), BAD), (dict(bias_f32=0, bias=FAR[2] + 1), BAD), (dict(bias_f32=2), BAD),
    (dict(residual=FAR[3] + 1), BAD), (dict(pre=FAR[5] + 1), BAD),
    (dict(x=FAR[0] + 2), BAD),                                    # restaged: workspace missing
    (dict(x=FAR[0] + 2, ws=FAR[6], ws_bytes=100), BAD),
    (dict(x=FAR[0] + 2, ws=FAR[6] + 128, ws_bytes=1 << 20), BAD),
    (dict(y=FAR[0] + 64), ALIAS), (dict(y=FAR[1] + 4096), ALIAS), (dict(y=FAR[2]), ALIAS),
    (dict(y=FAR[3], ldy=72), ALIAS), (dict(y=FAR[3] + 16), ALIAS), (dict(pre=FAR[4]), ALIAS),
    (dict(pre=FAR[3]), ALIAS), (dict(pre=FAR[0]), ALIAS),
    (dict(x=FAR[0] + 2, ws=FAR[4], ws_bytes=1 << 20), ALIAS),
    (dict(x=FAR[0] + 2, ws=FAR[1], ws_bytes=1 << 20), ALIAS)])
def test_refusals(lib, change, status):
    assert lib.gemm_bias_act(*args(LINEAR, change)) == status
    assert lib.tmm_last_error_string().decode()


GRAD = dict(dtype=_abi.TMM_BF16, transw=0, act=3, M=16, N=64, K=128, dy=FAR[0], lddy=64, x=FAR[1],
            ldx=128, w=FAR[2], ldw=64, pre=FAR[3], ldpre=64, dx=FAR[4], lddx=128, dw=FAR[5], lddw=64,
            transdw=0, dbias=FAR[6], ws=FAR[7], ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=-1), BAD), (dict(act=9), BAD), (dict(transdw=2), BAD), (dict(M=1 << 30), BAD),
    (dict(pre=0), BAD), (dict(dy=0), BAD), (dict(x=0), BAD), (dict(w=0), BAD),
    (dict(lddy=63), BAD), (dict(ldpre=1), BAD), (dict(lddx=127), BAD), (dict(lddw=63), BAD),
    (dict(transdw=1), BAD), (dict(dbias=FAR[6] + 2), BAD), (dict(ws=0), BAD),
    (dict(ws_bytes=16), BAD), (dict(ws=FAR[7] + 16), BAD),
    (dict(dx=FAR[0]), ALIAS), (dict(dw=FAR[1]), ALIAS), (dict(dbias=FAR[3]), ALIAS),
    (dict(dw=FAR[4]), ALIAS), (dict(ws=FAR[2]), ALIAS), (dict(ws=FAR[4]), ALIAS),
    (dict(dx=FAR[3] + 16), ALIAS)])
def test_gradient_refusals(lib, change, status):
    assert lib.gemm_bias_act_grad(*args(GRAD, change)) == status
    assert lib.tmm_last_error_string().decode()


def test_nothing_to_do_needs_no_device(lib):
    assert lib.gemm_bias_act(*args(LINEAR, dict(M=0))) == _abi.TMM_OK
    assert lib.gemm_bias_act(*args(LINEAR, dict(N=0, ldw=1, ldy=1))) == _abi.TMM_OK
    assert lib.gemm_bias_act_grad(*args(GRAD, dict(dx=0, dw=0, dbias=0))) == _abi.TMM_OK


@pytest.mark.parametrize("dtype,M,N,K", [(_abi.TMM_BF16, 16, 64, 128), (_abi.TMM_BF16, 1, 4096, 4096),
                                         (_abi.TMM_F16, 8192, 4096, 4096)])
def test_operands_on_16_byte_boundaries_need_no_workspace(lib, dtype, M, N, K):
    assert lib.gemm_bias_act_workspace_size(dtype, 0, M, N, K, FAR[0], K, FAR[1], N) == 0
    assert lib.gemm_bias_act_workspace_size(dtype, 1, M, N, K, FAR[0], K, FAR[1], K) == 0
    assert lib.gemm_bias_act_workspace_size(dtype, 0, M, N, K, FAR[0] + 2, K, FAR[1], N) > 0


@pytest.mark.parametrize("offset,ldw", [(0, 4096), (4, 4099)])
def test_few_rows_in_fp32_need_no_workspace(lib, offset, ldw):
    size = lib.gemm_bias_act_workspace_size
    assert all(size(_abi.TMM_F32, 0, M, 4096, 512, FAR[0] + offset, 512, FAR[1], ldw) == 0
               for M in (1, 5, 16))
    assert size(_abi.TMM_F32, 0, 17, 4096, 512, FAR[0] + offset, 512, FAR[1], ldw) >= 6 * 512 * 4096


def test_python_refusals():
    import tiled_matrix_multiply_gb300 as tmm
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        tmm.gemm_bias_act(x, x.t())
    with pytest.raises(TypeError):
        tmm.gemm_bias_act(x.double(), x.t().double())
    with pytest.raises(ValueError):
        tmm.gemm_bias_act_grad(x, x, x)


@pytest.mark.parametrize("kind", ref.ACTS)
def test_the_definitions_in_64_bits(kind):
    """The reference against torch's own functions."""
    torch_act = {"none": lambda z: z, "relu": torch.relu, "silu": torch.nn.functional.silu,
                 "gelu": torch.nn.functional.gelu,
                 "gelu_tanh": lambda z: torch.nn.functional.gelu(z, approximate="tanh")}[kind]
    gen = torch.Generator().manual_seed(1)
    z = (torch.randn(200, generator=gen, dtype=torch.float64) * 3).requires_grad_()
    y = torch_act(z)
    y.sum().backward()
    assert torch.allclose(ref.act(z.detach(), kind), y.detach(), atol=1e-12)
    assert torch.allclose(ref.slope(z.detach(), kind), z.grad, atol=1e-12)
