"""Grouped operators: products whose right-hand matrix is chosen row by row.

``group_rows`` sorts rows by a number each carries (its expert, its adapter);
``gemm_grouped`` multiplies every group's rows by that group's matrix (and, with
transposed views of the matrices, is the gradient with respect to the rows);
``gemm_grouped_wgrad`` is the gradient with respect to the matrices;
``gemm_lora`` adds every row's low-rank adapter to a shared projection.  Types
are bfloat16, float16 and float32, the same for all matrices of a call.

    plan = tmm.group_rows(experts, 8)               # experts: (tokens, k) integers
    h = tmm.gemm_grouped(x, w, plan.offsets, rows=plan.rows)        # (tokens * k, N)
    dw = tmm.gemm_grouped_wgrad(x, dh, plan.offsets, rows=plan.rows)
    dx_rows = tmm.gemm_grouped(dh, w.transpose(1, 2), plan.offsets)
    out = h[plan.position.view(tokens, k)]          # back in token order

Everything is asynchronous on the current torch stream of the operands' device (or, with
``stream``, on that stream, to which outputs and workspace then belong); no call reads a
group's size on the host.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
from typing import NamedTuple

import torch

from . import _abi, build as _build

_CODES = {torch.float32: _abi.TMM_F32, torch.bfloat16: _abi.TMM_BF16,
          torch.float16: _abi.TMM_F16}


class RowGroups(NamedTuple):
    """Slots sorted by group (see ``group_rows``), int32 CUDA tensors."""
    offsets: object     # (groups + 1): group g owns places offsets[g] .. offsets[g + 1] - 1
    order: object       # (slots): the slot at each place
    rows: object        # (slots): its token, order // k
    position: object    # (slots): the place of each slot


def _operand(x, name, like, dims, transposable=False):
    """(rows, cols, ld, stride, trans) of a matrix or a stack of matrices (dims = 3).

    stride: elements between matrices (0: one matrix, or an expanded one); trans = 1: every
    matrix is the transposed view of a row-major one, whose ld this is.
    """
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if x.dtype != like.dtype:
        raise TypeError(f"{name} must be {like.dtype} like the first operand, got {x.dtype}")
    if x.get_device() != like.get_device():
        raise ValueError(f"{name} is on {x.device}, the first operand on {like.device}")
    stride = 0
    if dims == 2:
        if x.dim() != 2:
            raise ValueError(f"{name} must be 2-D, got shape {tuple(x.shape)}")
        rows, cols = x.shape
        s0, s1 = x.stride()
    else:
        if x.dim() != 3:
            raise ValueError(f"{name} must be 3-D, got shape {tuple(x.shape)}")
        count, rows, cols = x.shape
        stride, s0, s1 = x.stride()
        if count <= 1:
            stride = 0
            if count == 0:
                return rows, cols, cols or 1, 0, 0
    if s1 == 1 and s0 >= cols:                       # the usual case
        return rows, cols, s0 or 1, stride, 0
    if rows == 0 or cols == 0:
        return rows, cols, cols or 1, stride, 0
    if (s1 == 1 or cols == 1) and (s0 >= cols or rows == 1):
        return rows, cols, max(s0 if rows > 1 else cols, cols), stride, 0
    if transposable and (s0 == 1 or rows == 1) and (s1 >= rows or cols == 1):
        return rows, cols, max(s1 if cols > 1 else rows, rows), stride, 1
    raise ValueError(f"{name} must be row-major (unit column stride)"
                     + (" or a transposed row-major view" if transposable else ""))


def _first(x, name):
    """The type code of the first operand, a matrix on a GPU."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    code = _CODES.get(x.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {x.dtype}")
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return code


def _index_ptr(t, name, like, length):
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32:
        raise TypeError(f"{name} must be an int32 tensor")
    if t.get_device() != like.get_device():
        raise ValueError(f"{name} is on {t.device}, the operands on {like.device}")
    if t.dim() != 1 or (length is not None and t.shape[0] != length) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 1-D tensor"
                         + (f" of {length} values" if length is not None else ""))
    return t.data_ptr()


def _result(given, name, shape, like):
    if given is None:
        return torch.empty(shape, dtype=like.dtype, device=like.device)
    if tuple(given.shape) != shape:
        raise ValueError(f"{name} must be {shape}, got {tuple(given.shape)}")
    return given


def _given_workspace(given, like):
    if not isinstance(given, torch.Tensor) or given.get_device() != like.get_device() \
            or not given.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the operands' device")
    return given


# The handle of the current stream of a device, without making a Stream object for it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda device: torch.cuda.current_stream(device).cuda_stream)


def _on_stream(stream, like, fn, *args, **kwargs):
    """The call with `stream` as the current one, so that what it allocates belongs there."""
    if stream.device != like.device:
        raise ValueError(f"stream is on {stream.device}, the operands on {like.device}")
    with torch.cuda.stream(stream):
        return fn(*args, **kwargs)


def _call(name, like, ws, *args):
    """Call the entry point on the operands' device and its current stream; raise its error."""
    device = like.get_device()
    s = _raw_stream(device)
    lib = _abi.load()
    if torch.cuda.current_device() == device:
        rc = _try(lib, name, ws, s, args)
    else:
        with torch.cuda.device(device):
            rc = _try(lib, name, ws, s, args)
    if rc != _abi.TMM_OK:
        raise _abi.TmmError(name, rc, _abi.last_error())


def _try(lib, name, ws, s, args):
    if ws is None:
        return getattr(lib, name)(*args, None, 0, s)
    return getattr(lib, name)(*args, ws.data_ptr(), ws.numel() * ws.element_size(), s)


def _scratch(need, like):
    """A workspace of `need` bytes, None for 0 (torch's blocks start on 512-byte boundaries)."""
    return torch.empty(need, dtype=torch.uint8, device=like.device) if need else None


class _NoCall:
    """In the marshalling module's place where it cannot be built: every call is an unusual one."""

    @staticmethod
    def group_rows(*_):
        return None

    grouped = wgrad = lora = group_rows


def _load_call():
    """The module that takes the usual calls (csrc/grouped_call.c), handed what it needs."""
    if not os.path.exists(_build.CALL_PATH):
        if not _build.call_buildable():
            return _NoCall
        raise RuntimeError(f"{_build.CALL_PATH} is missing: build it with "
                           "tiled_matrix_multiply_gb300.build.build()")
    loader = importlib.machinery.ExtensionFileLoader("grouped_call", _build.CALL_PATH)
    module = importlib.util.module_from_spec(
        importlib.util.spec_from_file_location("grouped_call", _build.CALL_PATH, loader=loader))
    loader.exec_module(module)
    lib = _abi.load()
    names = ("group_rows", "group_rows_workspace_size", "gemm_grouped",
             "gemm_grouped_workspace_size", "gemm_grouped_wgrad",
             "gemm_grouped_wgrad_workspace_size", "gemm_lora", "gemm_lora_workspace_size")
    module.start((torch.Tensor, torch.empty, _raw_stream, torch.cuda.current_device, RowGroups,
                  torch.uint8, torch.int32, torch.int64, torch.float32, torch.float32,
                  torch.bfloat16, torch.float16),
                 tuple(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in names))
    return module


_usual = _load_call()


def group_rows(index, groups, stream=None):
    """Stable grouping of the slots of ``index`` (tokens,) or (tokens, k), int32 or int64.

    A slot's group is its number where that is in [0, groups); the other slots belong to no
    group and come last.  Returns ``RowGroups``.
    """
    if stream is None:
        done = _usual.group_rows(index, groups)
        if done is not None:
            return done
    if not isinstance(index, torch.Tensor) or index.dtype not in (torch.int32, torch.int64):
        raise TypeError("index must be an int32 or int64 tensor")
    if not index.is_cuda:
        raise ValueError("index must be a CUDA tensor")
    if stream is not None:
        return _on_stream(stream, index, group_rows, index, groups)
    shape = index.shape
    if len(shape) not in (1, 2) or not index.is_contiguous():
        raise ValueError("index must be a contiguous tensor (tokens,) or (tokens, k)")
    tokens, fan = shape[0], shape[1] if len(shape) == 2 else 1
    if fan < 1:
        raise ValueError("index must have at least one column")
    if not 1 <= groups <= _abi.TMM_MAX_GROUPS:
        raise ValueError(f"groups must be between 1 and {_abi.TMM_MAX_GROUPS}, got {groups}")
    # (Four allocations: views of one cost three times as much to make.)
    i32, device, slots = torch.int32, index.device, tokens * fan
    offsets = torch.empty(groups + 1, dtype=i32, device=device)
    order = torch.empty(slots, dtype=i32, device=device)
    rows = torch.empty(slots, dtype=i32, device=device)
    position = torch.empty(slots, dtype=i32, device=device)
    ws = _scratch(_abi.load().group_rows_workspace_size(tokens, fan, groups), index)
    _call("group_rows", index, ws, tokens, fan, groups, index.data_ptr(),
          64 if index.dtype == torch.int64 else 32, offsets.data_ptr(), order.data_ptr(),
          rows.data_ptr(), position.data_ptr())
    return RowGroups(offsets, order, rows, position)


def gemm_grouped(x, w, offsets, rows=None, y=None, workspace=None, stream=None):
    """y[p] = x[rows[p]] w[g] for the rows p of every group g (offsets[g] <= p < offsets[g+1]).

    x: (x_rows, K); w: (groups, K, N), or a transposed view of (groups, N, K); offsets: int32
    (groups + 1); rows: int32, the row of x that each p reads (a number outside x reads zeros),
    or None for p itself.  y: (len(rows) or x_rows, N); its rows of no group are zero.
    """
    if y is None and workspace is None and stream is None:
        done = _usual.grouped(x, w, offsets, rows)
        if done is not None:
            return done
    code = _first(x, "x")
    if stream is not None:
        return _on_stream(stream, x, gemm_grouped, x, w, offsets, rows, y, workspace)
    x_rows, K, ldx, _, _ = _operand(x, "x", x, 2)
    K2, N, ldw, stride_w, trans = _operand(w, "w", x, 3, True)
    groups = w.shape[0]
    if K != K2:
        raise ValueError(f"inner dimensions differ: x is {tuple(x.shape)}, w is {tuple(w.shape)}")
    offsets_ptr = _index_ptr(offsets, "offsets", x, groups + 1)
    R, rows_ptr = x_rows, 0
    if rows is not None:
        rows_ptr = _index_ptr(rows, "rows", x, None)
        R = rows.shape[0]
    if y is None:
        y, ldy = torch.empty((R, N), dtype=x.dtype, device=x.device), N or 1
    else:
        ldy = _operand(_result(y, "y", (R, N), x), "y", x, 2)[2]
    w_ptr = w.data_ptr()
    head = (code, trans, groups, R, N, K, x.data_ptr(), x_rows, ldx)
    if workspace is None:
        workspace = _scratch(_abi.load().gemm_grouped_workspace_size(
            *head, rows_ptr, w_ptr, ldw, stride_w), x)
    else:
        _given_workspace(workspace, x)
    _call("gemm_grouped", x, workspace, *head, offsets_ptr, rows_ptr, w_ptr, ldw,
          stride_w, y.data_ptr(), ldy)
    return y


def gemm_grouped_wgrad(x, dy, offsets, rows=None, dw=None, workspace=None, stream=None):
    """dw[g] = sum over the rows p of group g of x[rows[p]]^T dy[p]: (groups, K, N).

    The gradient of ``gemm_grouped`` with respect to w; x, offsets and rows as there, dy (R, N).
    """
    if dw is None and workspace is None and stream is None:
        done = _usual.wgrad(x, dy, offsets, rows)
        if done is not None:
            return done
    code = _first(x, "x")
    if stream is not None:
        return _on_stream(stream, x, gemm_grouped_wgrad, x, dy, offsets, rows, dw, workspace)
    x_rows, K, ldx, _, _ = _operand(x, "x", x, 2)
    R, N, lddy, _, _ = _operand(dy, "dy", x, 2)
    offsets_ptr = _index_ptr(offsets, "offsets", x, None)
    groups = offsets.shape[0] - 1
    if groups < 1:
        raise ValueError("offsets must have groups + 1 values")
    rows_ptr = 0
    if rows is not None:
        rows_ptr = _index_ptr(rows, "rows", x, R)
    elif x_rows != R:
        raise ValueError(f"x has {x_rows} rows, dy {R}")
    dw = _result(dw, "dw", (groups, K, N), x)
    _, _, lddw, stride, _ = _operand(dw, "dw", x, 3)
    dy_ptr = dy.data_ptr()
    head = (code, groups, R, N, K, x.data_ptr(), x_rows, ldx)
    if workspace is None:
        workspace = _scratch(_abi.load().gemm_grouped_wgrad_workspace_size(
            *head, rows_ptr, dy_ptr, lddy), x)
    else:
        _given_workspace(workspace, x)
    _call("gemm_grouped_wgrad", x, workspace, *head, offsets_ptr, rows_ptr, dy_ptr, lddy,
          dw.data_ptr(), lddw, stride)
    return dw


def gemm_lora(x, w, a, b, scale, offsets, rows=None, y=None, workspace=None, stream=None):
    """y[t] = x[t] w + scale[g] (x[t] a[g]) b[g], g the adapter of row t.

    x: (T, K); w: (K, N); a: (adapters, K, r); b: (adapters, r, N) -- w, a and b also as
    transposed views; scale: float32 (adapters,).  offsets, rows: the rows grouped by adapter,
    ``offsets`` and ``order`` of ``group_rows(index, adapters)``; rows past offsets[-1] have no
    adapter.  rows=None: x is in group order already.  The product x[t] a[g] has FP32's range for
    every type; an infinite entry of b may give NaN where the formula gives an infinity.
    """
    if y is None and workspace is None and stream is None:
        done = _usual.lora(x, w, a, b, scale, offsets, rows)
        if done is not None:
            return done
    code = _first(x, "x")
    if stream is not None:
        return _on_stream(stream, x, gemm_lora, x, w, a, b, scale, offsets, rows, y, workspace)
    T, K, ldx, _, _ = _operand(x, "x", x, 2)
    K2, N, ldw, _, tw = _operand(w, "w", x, 2, True)
    K3, r, lda, stride_a, ta = _operand(a, "a", x, 3, True)
    r2, N2, ldb, stride_b, tb = _operand(b, "b", x, 3, True)
    groups = a.shape[0]
    if K != K2 or K != K3 or N != N2 or r != r2 or b.shape[0] != groups:
        raise ValueError(f"shapes do not fit: x {tuple(x.shape)}, w {tuple(w.shape)}, "
                         f"a {tuple(a.shape)}, b {tuple(b.shape)}")
    if not isinstance(scale, torch.Tensor) or scale.dtype != torch.float32:
        raise TypeError("scale must be a float32 tensor")
    if scale.dim() != 1 or scale.shape[0] != groups or scale.get_device() != x.get_device() \
            or not scale.is_contiguous():
        raise ValueError(f"scale must be a contiguous tensor of {groups} values on {x.device}")
    offsets_ptr = _index_ptr(offsets, "offsets", x, groups + 1)
    rows_ptr = _index_ptr(rows, "rows", x, T) if rows is not None else 0
    if y is None:
        y, ldy = torch.empty((T, N), dtype=x.dtype, device=x.device), N or 1
    else:
        ldy = _operand(_result(y, "y", (T, N), x), "y", x, 2)[2]
    head = (code, tw, ta, tb, groups, T, N, K, r, x.data_ptr(), ldx)
    mats = (w.data_ptr(), ldw, a.data_ptr(), lda, stride_a, b.data_ptr(), ldb, stride_b)
    if workspace is None:
        workspace = _scratch(_abi.load().gemm_lora_workspace_size(*head, rows_ptr, *mats), x)
    else:
        _given_workspace(workspace, x)
    _call("gemm_lora", x, workspace, *head, offsets_ptr, rows_ptr, *mats,
          scale.data_ptr(), y.data_ptr(), ldy)
    return y
