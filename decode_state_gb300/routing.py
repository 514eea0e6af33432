"""Routing: which k of n entries a token takes, and with which weights.

The entries are a stream's memory slots (the results are then ``k_idx`` / ``k_val`` or ``q_idx`` /
``q_val`` of a decode, or an operand of a gather) or experts (whose outputs a gather joins). The
definition, with ties, masks and groups, stands at ``sdm_route`` in ``include/sdm.h``.
"""

from __future__ import annotations

import torch

from . import sdm
from .sdm import _BANK_CODES, _IDX_CODES, _check, _need, _shape, _stream_handle

SCORES = {"softmax": 0, "sigmoid": 1}  # SDM_SOFTMAX, SDM_SIGMOID
SDM_RENORM = 4


def _row_stride(x: torch.Tensor, name: str, n: int) -> int:
    """Elements between rows of a [tokens, n] tensor with contiguous columns."""
    if x.dim() != 2:
        raise ValueError(f"{name} must be [tokens, n]")
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if x.dtype not in _BANK_CODES:
        raise TypeError(f"{name} must be bfloat16 or float32, got {x.dtype}")
    if x.is_contiguous():
        return n
    if n > 1 and x.stride(1) != 1 or x.shape[0] > 1 and x.stride(0) < n:
        raise ValueError(f"{name} must have contiguous columns and rows that do not overlap")
    return max(x.stride(0), n)


def _base(base, tokens: int, idx_dtype, dev):
    if base is None:
        return None
    _need(base, "base", dev)
    _shape(base, "base", (tokens,))
    if base.dtype != idx_dtype:
        raise TypeError(f"base must have the index dtype {idx_dtype}, got {base.dtype}")
    return base.data_ptr()


def _score(score: str) -> int:
    if score not in SCORES:
        raise ValueError(f"score must be one of {sorted(SCORES)}, got {score!r}")
    return SCORES[score]


def route(logits: torch.Tensor, k: int, *, score: str = "softmax", bias=None, groups: int = 1,
          top_groups: int | None = None, group_top: int = 1, renorm: bool = True, scale: float = 1.0, base=None,
          idx_dtype=torch.int32, idx=None, w=None, stream=None):
    """The k best entries of every row of ``logits`` [tokens, n] (bfloat16 or float32, rows by any
    stride), best first, and their weights: (idx [tokens, k], w [tokens, k] float32) (sdm_route).

    ``score`` "softmax" or "sigmoid"; ``bias`` [n] float32 is added to the scores for the choice
    only; with ``groups`` > 1 only the ``top_groups`` best groups take part (all when None), judged
    by their largest entry (``group_top`` 1) or the sum of their two largest (2); ``renorm`` divides
    the weights by their sum; ``scale`` multiplies them; ``base`` [tokens] is added to the indices
    (e.g. the first slot of the token's stream). Entries with a logit of -inf or NaN are masked."""
    tokens, n = logits.shape
    stride = _row_stride(logits, "logits", n)
    dev = logits.device
    if bias is not None:
        _need(bias, "bias", dev)
        sdm._f32(bias, "bias")
        _shape(bias, "bias", (n,))
    if idx is None:
        if idx_dtype not in _IDX_CODES:
            raise TypeError(f"indices must be int32 or int64, got {idx_dtype}")
        idx = torch.empty((tokens, k), dtype=idx_dtype, device=dev)
    else:
        _need(idx, "idx", dev)
        _shape(idx, "idx", (tokens, k))
        if idx.dtype not in _IDX_CODES:
            raise TypeError(f"idx must be int32 or int64, got {idx.dtype}")
    if w is None:
        w = torch.empty((tokens, k), dtype=torch.float32, device=dev)
    else:
        _need(w, "w", dev)
        _shape(w, "w", (tokens, k))
        sdm._f32(w, "w")
    rc = sdm.library().sdm_route(logits.data_ptr(), stride, _BANK_CODES[logits.dtype],
                                 None if bias is None else bias.data_ptr(), _base(base, tokens, idx.dtype, dev),
                                 idx.data_ptr(), w.data_ptr(), tokens, n, k, _score(score), groups,
                                 groups if top_groups is None else top_groups, group_top, scale,
                                 SDM_RENORM if renorm else 0, _IDX_CODES[idx.dtype], _stream_handle(stream, dev))
    _check("sdm_route", rc)
    return idx, w


def route_backward(logits: torch.Tensor, idx: torch.Tensor, dw: torch.Tensor, *, score: str = "softmax",
                   renorm: bool = True, scale: float = 1.0, base=None, out=None, stream=None) -> torch.Tensor:
    """Gradient of the logits from the gradient ``dw`` [tokens, k] (float32) of the weights, for the
    ``idx`` that ``route`` returned with the same ``score``, ``renorm``, ``scale`` and ``base``
    (sdm_route_backward). Returns [tokens, n] in the dtype of the logits."""
    tokens, n = logits.shape
    stride = _row_stride(logits, "logits", n)
    dev = logits.device
    _need(idx, "idx", dev)
    _need(dw, "dw", dev)
    if idx.dtype not in _IDX_CODES:
        raise TypeError(f"idx must be int32 or int64, got {idx.dtype}")
    sdm._f32(dw, "dw")
    k = idx.shape[-1]
    _shape(idx, "idx", (tokens, k))
    _shape(dw, "dw", (tokens, k))
    if out is None:
        out = torch.empty((tokens, n), dtype=logits.dtype, device=dev)
    elif out.dtype != logits.dtype or out.device != dev:
        raise TypeError("out must have the dtype and the device of the logits")
    _shape(out, "out", (tokens, n))
    rc = sdm.library().sdm_route_backward(logits.data_ptr(), stride, _BANK_CODES[logits.dtype],
                                          _base(base, tokens, idx.dtype, dev), idx.data_ptr(), dw.data_ptr(),
                                          out.data_ptr(), _row_stride(out, "out", n), tokens, n, k, _score(score),
                                          scale, SDM_RENORM if renorm else 0, _IDX_CODES[idx.dtype],
                                          _stream_handle(stream, dev))
    _check("sdm_route_backward", rc)
    return out
