"""The device status: bits of every operator's kernels, read once and reset, or left."""

from __future__ import annotations

import threading

import pytest
import torch

from decode_state_gb300 import quant, routing, sdm

pytestmark = pytest.mark.gpu


def _raising():
    """A call of each operator that meets an index outside its bank (or row), for either of its kernels."""
    rows = torch.ones(64, 32, device="cuda")
    bank = quant.QuantBank.from_rows(rows, group=32)
    one = torch.full((1,), 64, device="cuda")

    def pair(tokens):
        return torch.full((tokens, 4), 64, device="cuda"), torch.ones(tokens, 4, device="cuda")

    step = (torch.full((2, 4), 64, device="cuda"), torch.ones(2, 4, device="cuda"), torch.ones(2, 32, device="cuda"),
            torch.ones(2, device="cuda"), torch.zeros(2, 1, device="cuda"), torch.zeros((2, 4), dtype=torch.int64, device="cuda"),
            torch.ones(2, 4, device="cuda"))
    return {
        "gather": lambda: sdm.gather(rows, [pair(8)], chunk=1, with_stash=False),
        "quantize_rows": lambda: quant.quantize_rows(bank, rows[:1], one),
        "dequantize_rows": lambda: quant.dequantize_rows(bank, one),
        "qgather": lambda: quant.gather(bank, [pair(8)]),
        "qgather of many": lambda: quant.gather(bank, [pair(5000)]),
        "gather_dw": lambda: quant.gather_dw(bank, [(pair(8)[0], torch.ones(8, 32, device="cuda"))]),
        "qdecode": lambda: quant.decode_step(bank, *step),
        "route_backward": lambda: routing.route_backward(rows, torch.full((64, 1), 99, device="cuda"), torch.ones(64, 1, device="cuda")),
    }


def test_every_operator_raises_and_is_reset():
    sdm.device_status()
    for name, call in _raising().items():
        side = torch.cuda.Stream()  # a stream that does not block the default one
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call()
        assert sdm.device_status(clear=False) == sdm.SDM_DEV_BAD_INDEX, name
        assert sdm.device_status() == sdm.SDM_DEV_BAD_INDEX, name
        assert sdm.device_status() == 0, name


def test_threads_at_once():
    """Each bit is read once: the threads' words together have it, and then nobody's."""
    sdm.device_status()
    for _ in range(20):
        quant.dequantize_rows(quant.QuantBank.zeros(4, 32, group=32), torch.full((1,), 9, device="cuda"))
        got = []
        threads = [threading.Thread(target=lambda: got.append(sdm.device_status())) for _ in range(8)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert sorted(got) == [0] * 7 + [sdm.SDM_DEV_BAD_INDEX]
