"""Linear layers: a product with bias, activation and residual in its epilogue, and its gradients.

``gemm_bias_act`` is y = act(x w + bias) + residual in one kernel; ``gemm_bias_act_grad`` gives the
gradients with respect to x, w and bias.  Types are bfloat16, float16 and float32, the same for all
matrices of a call; the bias may be float32 beside 16-bit ones.  w is (K, N), or a transposed view of
(N, K) rows, which is how many frameworks keep a layer's weights.

    y, z = tmm.gemm_bias_act(x, weight.t(), bias, act="gelu", residual=x, pre=True)
    g = tmm.gemm_bias_act_grad(dy, x, weight.t(), pre=z, act="gelu", dbias=True)
    # g.dx, g.dw (laid out like weight.t()), g.dbias; the residual's gradient is dy

Everything is asynchronous on the current torch stream of the operands' device (or, with ``stream``,
on that stream, to which outputs and workspace then belong).
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import _abi
from .grouped import (_addresses, _call, _first, _given_workspace, _on_stream, _operand, _result,
                      _scratch, _usual)

_ACTS = {"none": _abi.TMM_ACT_NONE, "relu": _abi.TMM_ACT_RELU, "silu": _abi.TMM_ACT_SILU,
         "gelu": _abi.TMM_ACT_GELU, "gelu_tanh": _abi.TMM_ACT_GELU_TANH}


class LinearGrads(NamedTuple):
    """Gradients of ``gemm_bias_act``; None where not asked for."""
    dx: object
    dw: object
    dbias: object       # float32


_usual.start_linear((LinearGrads,), _addresses(
    "gemm_bias_act", "gemm_bias_act_workspace_size", "gemm_bias_act_grad",
    "gemm_bias_act_grad_workspace_size"))


def _act(act):
    code = _ACTS.get(act)
    if code is None:
        raise ValueError(f"act must be one of {', '.join(_ACTS)}, got {act!r}")
    return code


def _side(m, name, shape, like):
    """(address, ld) of a matrix of the result's shape."""
    if tuple(m.shape) != shape:
        raise ValueError(f"{name} must be {shape}, got {tuple(m.shape)}")
    ld = _operand(m, name, like, 2)[2]
    return m.data_ptr(), ld


def gemm_bias_act(x, w, bias=None, act="none", residual=None, y=None, pre=None, workspace=None,
                  stream=None):
    """y = act(x w + bias) + residual: x (M, K); w (K, N), also as a transposed view.

    bias: (N), of x's type or float32; act: "none", "relu", "silu", "gelu" or "gelu_tanh"; residual:
    (M, N), which y may be itself.  pre: True, or a matrix (M, N), to keep z = x w + bias for the
    gradients; then (y, z) is returned.
    """
    if y is None and workspace is None and stream is None:
        done = _usual.linear(x, w, bias, _ACTS.get(act, -1), residual, pre)
        if done is not None:
            return done
    code = _first(x, "x")
    if stream is not None:
        return _on_stream(stream, x, gemm_bias_act, x, w, bias, act, residual, y, pre, workspace)
    M, K, ldx, _, _ = _operand(x, "x", x, 2)
    K2, N, ldw, _, trans = _operand(w, "w", x, 2, True)
    if K != K2:
        raise ValueError(f"inner dimensions differ: x is {tuple(x.shape)}, w is {tuple(w.shape)}")
    bias_ptr, bias_f32 = 0, 0
    if bias is not None:
        if not isinstance(bias, torch.Tensor) or bias.dtype not in (x.dtype, torch.float32):
            raise TypeError(f"bias must be a {x.dtype} or float32 tensor")
        if tuple(bias.shape) != (N,) or not bias.is_contiguous() \
                or bias.get_device() != x.get_device():
            raise ValueError(f"bias must be a contiguous tensor of {N} values on {x.device}")
        bias_ptr, bias_f32 = bias.data_ptr(), int(bias.dtype == torch.float32)
    shape = (M, N)
    res_ptr, ldr = (0, 1) if residual is None else _side(residual, "residual", shape, x)
    if y is None:
        y, ldy = torch.empty(shape, dtype=x.dtype, device=x.device), N or 1
    else:
        ldy = _side(y, "y", shape, x)[1]
    z = pre
    if pre is True:
        z = torch.empty(shape, dtype=x.dtype, device=x.device)
    elif pre is False:
        z = None
    pre_ptr, ldp = (0, 1) if z is None else _side(z, "pre", shape, x)
    mats = (x.data_ptr(), ldx, w.data_ptr(), ldw)
    if workspace is None:
        workspace = _scratch(_abi.load().gemm_bias_act_workspace_size(code, trans, M, N, K, *mats), x)
    else:
        _given_workspace(workspace, x)
    _call("gemm_bias_act", x, workspace, code, trans, _act(act), M, N, K, *mats, bias_ptr, bias_f32,
          res_ptr, ldr, y.data_ptr(), ldy, pre_ptr, ldp)
    return y if z is None else (y, z)


def _wanted(given, shape, like, dtype=None):
    """A result: a given tensor, a new one for True, none for False or None."""
    if given is None or given is False:
        return None
    if given is True:
        return torch.empty(shape, dtype=dtype or like.dtype, device=like.device)
    return given


def gemm_bias_act_grad(dy, x, w, pre=None, act="none", dx=True, dw=True, dbias=False,
                       workspace=None, stream=None):
    """Gradients of ``gemm_bias_act`` from dy (M, N), as ``LinearGrads``.

    dz = dy act'(pre); dx = dz w^T, dw = x^T dz, dbias the sum of dz's rows in float32 (the
    residual's gradient is dy).  dz is rounded to the type's bits for the products, in float16 without
    that type's range.  pre: what ``gemm_bias_act`` kept (act "none" needs none).  dx, dw and dbias:
    True, False, or a tensor for the result; a new dw is laid out as w is.  w may be None without dx,
    and x without dw.
    """
    if dx is True and dw is True and workspace is None and stream is None:
        done = _usual.linear_grad(dy, x, w, pre, _ACTS.get(act, -1), dbias)
        if done is not None:
            return done
    code = _first(dy, "dy")
    if stream is not None:
        return _on_stream(stream, dy, gemm_bias_act_grad, dy, x, w, pre, act, dx, dw, dbias,
                          workspace)
    act_code = _act(act)
    M, N, lddy, _, _ = _operand(dy, "dy", dy, 2)
    x_ptr, ldx, w_ptr, ldw, trans, K = 0, 1, 0, 1, 0, None
    if x is not None:
        Mx, K, ldx, _, _ = _operand(x, "x", dy, 2)
        x_ptr = x.data_ptr()
        if Mx != M:
            raise ValueError(f"x is {tuple(x.shape)}, dy {tuple(dy.shape)}")
    if w is not None:
        Kw, Nw, ldw, _, trans = _operand(w, "w", dy, 2, True)
        w_ptr = w.data_ptr()
        if Nw != N or (K is not None and Kw != K):
            raise ValueError(f"w is {tuple(w.shape)}, dy {tuple(dy.shape)}"
                             + (f", x {tuple(x.shape)}" if x is not None else ""))
        K = Kw
    if (w is None and dx is not None and dx is not False) \
            or (x is None and dw is not None and dw is not False):
        raise ValueError("dx needs w and dw needs x")
    K = K or 0
    pre_ptr, ldp = 0, 1
    if act_code != _abi.TMM_ACT_NONE:
        if pre is None:
            raise ValueError(f"pre is needed for the gradient of {act!r}")
        pre_ptr, ldp = _side(pre, "pre", (M, N), dy)
    dx = _wanted(dx, (M, K), dy)
    dx_ptr, lddx = (0, 1) if dx is None else _side(dx, "dx", (M, K), dy)
    dw_ptr, lddw, trans_dw = 0, 1, 0
    if dw is True and trans:
        dw = torch.empty((N, K), dtype=dy.dtype, device=dy.device).t()
    dw = _wanted(dw, (K, N), dy)
    if dw is not None:
        _, _, lddw, _, trans_dw = _operand(_result(dw, "dw", (K, N), dy), "dw", dy, 2, True)
        dw_ptr = dw.data_ptr()
    dbias = _wanted(dbias, (N,), dy, torch.float32)
    if dbias is not None:
        if not isinstance(dbias, torch.Tensor) or dbias.dtype != torch.float32:
            raise TypeError("dbias must be a float32 tensor")
        if tuple(dbias.shape) != (N,) or not dbias.is_contiguous() \
                or dbias.get_device() != dy.get_device():
            raise ValueError(f"dbias must be a contiguous tensor of {N} values on {dy.device}")
    bias_ptr = 0 if dbias is None else dbias.data_ptr()
    head = (code, trans, act_code, M, N, K, dy.data_ptr(), lddy, x_ptr, ldx, w_ptr, ldw)
    if workspace is None:
        workspace = _scratch(_abi.load().gemm_bias_act_grad_workspace_size(
            *head, dx_ptr, dw_ptr, trans_dw, bias_ptr), dy)
    else:
        _given_workspace(workspace, dy)
    _call("gemm_bias_act_grad", dy, workspace, *head, pre_ptr, ldp, dx_ptr, lddx, dw_ptr, lddw,
          trans_dw, bias_ptr)
    return LinearGrads(dx, dw, dbias)
