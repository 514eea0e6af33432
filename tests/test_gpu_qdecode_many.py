"""Decode on quantised banks with more blocks than two for each multiprocessor, where blocks have fewer
threads: the checks and tolerances of the small cases, and the same bits from both call forms."""

from __future__ import annotations

import pytest
import test_gpu_quant as small

from decode_state_gb300 import sdm

pytestmark = pytest.mark.gpu

MANY = [(310, 40, 128, 64, 20, 20, 1, 2), (320, 90, 128, 128, 64, 64, 64, 2), (160, 90, 200, 64, 50, 33, 1, 2),
        (400, 70, 40, 32, 64, 5, 1, 2), (306, 70, 64, 64, 9, 200, 9, 2), (305, 140, 128, 32, 128, 128, 1, 1),
        (305, 30, 16, 32, 3, 1, 1, 3)]


@pytest.fixture(autouse=True)
def _clean_status():
    sdm.device_status()
    yield
    assert sdm.device_status() == 0


@pytest.mark.parametrize("fmt", ("int8", "fp8"))
@pytest.mark.parametrize("S,P,hd,group,W,R,G,T", MANY)
def test_decode_of_many_streams(fmt, S, P, hd, group, W, R, G, T):
    small.test_decode(fmt, S, P, hd, group, W, R, G, T)


@pytest.mark.parametrize("fmt", ("int8", "fp8"))
@pytest.mark.parametrize("S,P,hd,group,W,R,G,T", [(330, 80, 128, 64, 64, 64, 1, 5), (320, 50, 60, 32, 30, 17, 30, 4),
                                                  (3, 300, 128, 64, 256, 256, 1, 4)])
def test_steps_and_sequence(fmt, S, P, hd, group, W, R, G, T):
    small.test_decode_seq_is_the_steps(fmt, S, P, hd, group, W, R, G, T)
