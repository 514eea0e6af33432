"""Routing: which k of n entries a token takes, and with which weights.

The entries are a stream's memory slots (the results are then ``k_idx`` / ``k_val`` or ``q_idx`` /
``q_val`` of a decode, or an operand of a gather) or experts (whose outputs a gather joins). The
definition, with ties, masks and groups, stands at ``sdm_route`` in ``include/sdm.h``. Work goes to the
current stream unless ``stream`` is given; outputs are then made in that stream's memory.
"""

from __future__ import annotations

import torch

from .sdm import binding

SCORES = {"softmax": 0, "sigmoid": 1}  # SDM_SOFTMAX, SDM_SIGMOID


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
    return binding().route(logits, k, _score(score), bias, groups, groups if top_groups is None else top_groups, group_top,
                           renorm, scale, base, idx_dtype, idx, w, stream)


def route_backward(logits: torch.Tensor, idx: torch.Tensor, dw: torch.Tensor, *, score: str = "softmax",
                   renorm: bool = True, scale: float = 1.0, base=None, w=None, out=None, stream=None) -> torch.Tensor:
    """Gradient of the logits from the gradient ``dw`` [tokens, k] (float32) of the weights, for the
    ``idx`` that ``route`` returned with the same ``score``, ``renorm``, ``scale`` and ``base``
    (sdm_route_backward_ex). Returns [tokens, n] in the dtype of the logits.

    ``w``, the weights that ``route`` returned, tells which entries only filled up: those of weight 0
    have no gradient. It is needed wherever ``groups`` or a ``bias`` of -inf may leave fewer than k
    entries; without it every entry with a live logit is taken as chosen."""
    return binding().route_backward(logits, idx, dw, _score(score), renorm, scale, base, w, out, stream)
