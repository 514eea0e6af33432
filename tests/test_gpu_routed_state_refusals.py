"""What the routed decode state refuses: rows that do not fill the bank, logits that are no single reading."""

from __future__ import annotations

import pytest
import torch

from decode_state_gb300 import quant
from decode_state_gb300.state import RoutedLayerState

pytestmark = pytest.mark.gpu


def _state():
    return RoutedLayerState(quant.QuantBank.from_rows(torch.ones(20, 32, device="cuda"), group=32), 4, writes=2, reads=2)


@pytest.mark.parametrize("rows", (0, 1, 19, 21))
def test_load_takes_all_rows(rows):
    s = _state()
    with pytest.raises(ValueError):
        s.load_(torch.zeros(rows, 32, device="cuda"), 3)
    assert s.cache_len == 0 and (s.rows() != 0).all()  # the state is as it was


def test_read_takes_one_reading():
    s = _state()
    q = torch.randn(3, 4, 5, device="cuda")
    with pytest.raises(ValueError, match="logits must be"):
        s.read(q)
    out, idx, w = s.read(q[0])
    with pytest.raises(ValueError, match="logits must be"):
        s.read_backward(q, idx, out)
