"""Embedding rows: scaled rows of a table by token, and the gradient of the table.

Tables are [rows, hd] bfloat16 or float32, tokens int32 or int64 of any shape, all of them contiguous. ``padding`` names a token that stands for
nothing: it gives zeros and has no gradient. A token outside the table does likewise and raises the device status
(``sdm.device_status``). Work goes to the current stream unless ``stream`` is given; outputs are then made in that
stream's memory. The definitions stand at ``sdm_lookup`` and ``sdm_lookup_backward`` in ``include/sdm.h``.
"""

from __future__ import annotations

import torch

from .sdm import binding


def lookup(table: torch.Tensor, tokens: torch.Tensor, *, scale: float = 1.0, padding: int | None = None, dtype=None, out=None,
           stream=None) -> torch.Tensor:
    """``scale`` times the tokens' rows, [*tokens.shape, hd] in ``dtype`` (the table's when None), rounded once."""
    return binding().lookup(table, tokens, scale, padding, dtype, out, stream)


def backward(dout: torch.Tensor, tokens: torch.Tensor, rows: int, *, scale: float = 1.0, padding: int | None = None,
             dtype=torch.float32, out=None, accumulate: bool = False, stream=None) -> torch.Tensor:
    """Gradient [rows, hd] of the table of ``lookup`` from that of its output, ``dout`` [*tokens.shape, hd] (bfloat16 or
    float32): ``scale`` times the sums of dout by token, in float32 and rounded to ``dtype`` once. ``out`` gives the
    tensor to write, and with ``accumulate`` the tensor to add to, of which only the tokens' rows are touched."""
    return binding().lookup_backward(dout, tokens, rows, scale, padding, dtype, out, accumulate, stream)
