"""What the routed decode state refuses before it touches a GPU."""

from __future__ import annotations

from types import SimpleNamespace

import pytest
import torch

from decode_state_gb300.state import RoutedLayerState


def _bank(n_slots=12):
    return SimpleNamespace(n_slots=n_slots, device=torch.device("cpu"), hd=8)


def test_slots_divide_among_streams():
    assert RoutedLayerState(_bank(), 3, writes=2, reads=2, seq_len=5).cache_len == 5
    for streams in (0, -1, 5):
        with pytest.raises(ValueError, match="do not divide"):
            RoutedLayerState(_bank(), streams, writes=2, reads=2)


@pytest.mark.parametrize("name", ("base", "idx_dtype", "idx", "w", "stream"))
def test_arguments_that_the_state_sets(name):
    with pytest.raises(ValueError, match=f"{name} is set by the state"):
        RoutedLayerState(_bank(), 3, writes=2, reads=2, **{name: None})


@pytest.mark.parametrize("shape", ((3, 5), (4, 4), (2, 3, 3), (12,)))
def test_logits_of_other_shapes(shape):
    with pytest.raises(ValueError, match="logits must be"):
        RoutedLayerState(_bank(), 3, writes=2, reads=2).choose(torch.zeros(shape), 2)
