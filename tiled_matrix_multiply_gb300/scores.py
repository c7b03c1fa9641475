"""Operators over rows of scores: routing to experts, and log probabilities.

``route_rows`` chooses every token's experts and their weights from a router's logits, and
``group_rows`` sorts what it chose for the grouped products; ``logprob_rows`` gives the log
probabilities of given tokens, the entropies and the most probable tokens under rows of logits.
``route_rows_grad`` and ``logprob_rows_grad`` are their gradients.  Logits are bfloat16, float16 or
float32 matrices with any row stride; probabilities and weights are float32.

    r = tmm.route_rows(logits, 8, bias=balance, score="sigmoid", groups=8, top_groups=4,
                       group_best=2)
    plan = tmm.group_rows(r.experts, logits.shape[1])
    ...
    dlogits = tmm.route_rows_grad(dweights, logits, r.experts, score="sigmoid")

    p = tmm.logprob_rows(logits, tokens, top=5)
    dlogits = tmm.logprob_rows_grad(logits, tokens, p.lse, dlogprob=g)

Everything is asynchronous on the current torch stream of the logits' device (or, with ``stream``, on
that stream, to which outputs then belong).
"""
from __future__ import annotations

import math
from typing import NamedTuple

import torch

from . import _abi
from .grouped import _addresses, _call_plain, _first, _on_stream, _operand, _usual

_SCORES = {"softmax": _abi.TMM_SOFTMAX, "sigmoid": _abi.TMM_SIGMOID}


class RowRoutes(NamedTuple):
    """What every token's row goes to (see ``route_rows``), CUDA tensors (tokens, k)."""
    experts: object     # int32: the experts, best first; -1 where none was left
    weights: object     # float32


class RowLogprobs(NamedTuple):
    """Log probabilities of rows of logits (see ``logprob_rows``), float32 CUDA tensors."""
    logprob: object        # (rows): of the given token, or None without tokens
    entropy: object        # (rows)
    lse: object            # (rows): log of the sum of exponentials
    top_ids: object        # int32 (rows, top), or None
    top_logprobs: object   # (rows, top), or None


_usual.start_scores((RowRoutes, RowLogprobs),
                    _addresses("route_rows", "route_rows_grad", "logprob_rows",
                               "logprob_rows_grad"))


def _score(score):
    code = _SCORES.get(score)
    if code is None:
        raise ValueError(f'score must be "softmax" or "sigmoid", got {score!r}')
    return code


def _vector(t, name, like, shape, dtypes=(torch.float32,)):
    """The address of a contiguous tensor beside the logits."""
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes:
        raise TypeError(f"{name} must be a {' or '.join(str(d) for d in dtypes)} tensor")
    if t.get_device() != like.get_device():
        raise ValueError(f"{name} is on {t.device}, the logits on {like.device}")
    if tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of shape {shape}, got "
                         f"{tuple(t.shape)}")
    return t.data_ptr()


def _finite(scale, positive=False):
    scale = float(scale)
    if not math.isfinite(scale) or (positive and scale <= 0):
        raise ValueError(f"scale must be finite{' and positive' if positive else ''}, got {scale}")
    return scale


def _like_logits(out, logits, name):
    """The result of a gradient call: given (logits itself for a call in place) or new."""
    if out is None:
        out = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
    elif tuple(out.shape) != tuple(logits.shape):
        raise ValueError(f"{name} must be {tuple(logits.shape)}, got {tuple(out.shape)}")
    return out, _operand(out, name, logits, 2)[2]


def route_rows(logits, k, bias=None, score="softmax", groups=1, top_groups=1, group_best=1,
               renormalise=True, scale=1.0, stream=None):
    """The ``k`` best experts of every row of ``logits`` (tokens, experts), as ``RowRoutes``.

    s = softmax or sigmoid of the logits; c = s + bias (float32 (experts), a bias for balance that
    moves the choice and not the weights).  Only experts of the ``top_groups`` best of ``groups``
    equal groups are chosen, a group's value being the sum of its ``group_best`` (1 or 2) largest c;
    ties go to the lower number.  weights = scale * s / (sum of the chosen s), without
    ``renormalise`` scale * s.  An expert whose logit or bias is -inf is never chosen; where none is
    left the expert is -1 and its weight 0.  A row with NaN or +inf has NaN weights under the softmax,
    at whichever expert; under sigmoids one with NaN at an expert whose bias is not -inf.
    """
    if stream is None:
        done = _usual.route(logits, k, bias, _SCORES.get(score, -1), groups, top_groups, group_best,
                            renormalise, scale)
        if done is not None:
            return done
    code = _first(logits, "logits")
    if stream is not None:
        return _on_stream(stream, logits, route_rows, logits, k, bias, score, groups, top_groups,
                          group_best, renormalise, scale)
    tokens, experts, ld, _, _ = _operand(logits, "logits", logits, 2)
    if not 1 <= k <= _abi.TMM_MAX_FAN:
        raise ValueError(f"k must be between 1 and {_abi.TMM_MAX_FAN}, got {k}")
    bias_ptr = 0 if bias is None else _vector(bias, "bias", logits, (experts,))
    chosen = torch.empty((tokens, k), dtype=torch.int32, device=logits.device)
    weights = torch.empty((tokens, k), dtype=torch.float32, device=logits.device)
    _call_plain("route_rows", logits, code, tokens, experts, logits.data_ptr(), ld, bias_ptr,
                _score(score), groups, top_groups, group_best, k, int(bool(renormalise)),
                _finite(scale), chosen.data_ptr(), weights.data_ptr())
    return RowRoutes(chosen, weights)


def route_rows_grad(dweights, logits, experts, score="softmax", renormalise=True, scale=1.0,
                    dlogits=None, stream=None):
    """The gradient of ``route_rows``' weights with respect to the logits, the choice held fixed.

    dweights: float32 (tokens, k); logits, score, renormalise and scale as there; experts: int32
    (tokens, k), what it chose (numbers outside the experts have no part).  dlogits may be logits.
    """
    if dlogits is None and stream is None:
        done = _usual.route_grad(dweights, logits, experts, _SCORES.get(score, -1), renormalise,
                                 scale)
        if done is not None:
            return done
    code = _first(logits, "logits")
    if stream is not None:
        return _on_stream(stream, logits, route_rows_grad, dweights, logits, experts, score,
                          renormalise, scale, dlogits)
    tokens, count, ld, _, _ = _operand(logits, "logits", logits, 2)
    if not isinstance(dweights, torch.Tensor) or dweights.dim() != 2:
        raise TypeError("dweights must be a 2-D tensor")
    k = dweights.shape[1]
    shape = (tokens, k)
    dw_ptr = _vector(dweights, "dweights", logits, shape)
    chosen_ptr = _vector(experts, "experts", logits, shape, (torch.int32,))
    dlogits, ldd = _like_logits(dlogits, logits, "dlogits")
    _call_plain("route_rows_grad", logits, code, tokens, count, k, dw_ptr, logits.data_ptr(), ld,
                chosen_ptr, _score(score), int(bool(renormalise)), _finite(scale),
                dlogits.data_ptr(), ldd)
    return dlogits


def _tokens(tokens, logits, rows):
    """(address, bits) of the given tokens."""
    ptr = _vector(tokens, "tokens", logits, (rows,), (torch.int64, torch.int32))
    return ptr, 64 if tokens.dtype == torch.int64 else 32


def logprob_rows(logits, tokens=None, top=0, scale=1.0, stream=None):
    """Log probabilities under the softmax of every row of ``scale * logits`` (rows, vocabulary).

    tokens: int64 or int32 (rows), each row's given token (outside the vocabulary, padding: its log
    probability is 0, whatever the row's logits), or None.  top: how many of the most probable tokens
    to list, at most 32.  Returns ``RowLogprobs``.
    """
    if stream is None:
        done = _usual.logprob(logits, tokens, top, scale)
        if done is not None:
            return done
    code = _first(logits, "logits")
    if stream is not None:
        return _on_stream(stream, logits, logprob_rows, logits, tokens, top, scale)
    rows, cols, ld, _, _ = _operand(logits, "logits", logits, 2)
    if not 0 <= top <= _abi.TMM_MAX_TOP:
        raise ValueError(f"top must be between 0 and {_abi.TMM_MAX_TOP}, got {top}")
    ptr, bits = (0, 32) if tokens is None else _tokens(tokens, logits, rows)

    def new(*shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device=logits.device)

    logprob = None if tokens is None else new(rows)
    entropy, lse = new(rows), new(rows)
    ids, of_ids = (new(rows, top, dtype=torch.int32), new(rows, top)) if top else (None, None)
    _call_plain("logprob_rows", logits, code, rows, cols, logits.data_ptr(), ld,
                _finite(scale, True), ptr, bits, top, logprob.data_ptr() if tokens is not None else 0,
                entropy.data_ptr(), lse.data_ptr(), ids.data_ptr() if top else 0,
                of_ids.data_ptr() if top else 0)
    return RowLogprobs(logprob, entropy, lse, ids, of_ids)


def logprob_rows_grad(logits, tokens, lse, dlogprob=None, entropy=None, dentropy=None, top_ids=None,
                      dtop=None, scale=1.0, dlogits=None, stream=None):
    """The gradient of ``logprob_rows`` with respect to the logits (rows, vocabulary).

    lse, and for their gradients entropy and top_ids, as ``logprob_rows`` gave them; dlogprob (with
    tokens), dentropy: float32 (rows); dtop: float32 (rows, top), the gradient of the listed log
    probabilities.  dlogits may be logits (in place).
    """
    if dlogits is None and stream is None:
        done = _usual.logprob_grad(logits, tokens, lse, dlogprob, entropy, dentropy, top_ids, dtop,
                                   scale)
        if done is not None:
            return done
    code = _first(logits, "logits")
    if stream is not None:
        return _on_stream(stream, logits, logprob_rows_grad, logits, tokens, lse, dlogprob, entropy,
                          dentropy, top_ids, dtop, scale, dlogits)
    rows, cols, ld, _, _ = _operand(logits, "logits", logits, 2)
    lse_ptr = _vector(lse, "lse", logits, (rows,))
    tok_ptr, bits, g_ptr, h_ptr, entropy_ptr = 0, 32, 0, 0, 0
    if dlogprob is not None:
        tok_ptr, bits = _tokens(tokens, logits, rows)
        g_ptr = _vector(dlogprob, "dlogprob", logits, (rows,))
    if dentropy is not None:
        h_ptr = _vector(dentropy, "dentropy", logits, (rows,))
        entropy_ptr = _vector(entropy, "entropy", logits, (rows,))
    top, ids_ptr, dtop_ptr = 0, 0, 0
    if dtop is not None:
        if not isinstance(dtop, torch.Tensor) or dtop.dim() != 2:
            raise TypeError("dtop must be a 2-D tensor")
        top = dtop.shape[1]
        dtop_ptr = _vector(dtop, "dtop", logits, (rows, top))
        ids_ptr = _vector(top_ids, "top_ids", logits, (rows, top), (torch.int32,))
    dlogits, ldd = _like_logits(dlogits, logits, "dlogits")
    _call_plain("logprob_rows_grad", logits, code, rows, cols, logits.data_ptr(), ld,
                _finite(scale, True), lse_ptr, tok_ptr, bits, g_ptr, entropy_ptr, h_ptr, top,
                ids_ptr, dtop_ptr, dlogits.data_ptr(), ldd)
    return dlogits
