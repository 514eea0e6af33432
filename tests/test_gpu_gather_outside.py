"""Entries whose index lies outside the bank are skipped: their weight (or the gradient that comes to them), which
may be an infinity or NaN, changes nothing, and their own gradient is zero."""

from __future__ import annotations

import pytest
import torch

from decode_state_gb300 import quant, sdm

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


def _bank(hd, format, n_slots=500):
    rows = torch.randn((n_slots, hd), generator=torch.Generator().manual_seed(hd)).cuda()
    if format in ("bf16", "f32"):
        return rows.to(torch.bfloat16 if format == "bf16" else torch.float32)
    return quant.QuantBank.from_rows(rows, group=64, format=format)


def _entries(tokens, width, seed):
    """Indices of which about a tenth lie outside; one token has none inside, one none outside."""
    gen = torch.Generator().manual_seed(seed)
    idx = torch.randint(0, 500, (tokens, width), generator=gen)
    out = torch.rand((tokens, width), generator=gen) < 0.1
    out[0], out[1] = True, False
    idx[out] = torch.tensor([-1, 500, 1 << 30])[torch.arange(int(out.sum())) % 3]
    return idx, out, gen


@pytest.mark.parametrize("tokens", (9, 5000))
@pytest.mark.parametrize("hd,width", [(64, 7), (72, 40), (200, 33), (264, 5)])
@pytest.mark.parametrize("format", ("int8", "fp8", "int4"))
def test_weights(tokens, hd, width, format):
    idx, out, gen = _entries(tokens, width, hd + tokens)
    w = torch.randn((tokens, width), generator=gen)
    bad = w.clone()
    w[out] = 0.0
    bad[out] = torch.tensor([NAN, INF, -INF])[torch.arange(int(out.sum())) % 3]
    bank = _bank(hd, format)
    for dtype in (torch.float32, torch.bfloat16):
        want, = quant.gather(bank, [(idx.cuda(), w.cuda().to(dtype))])
        got, = quant.gather(bank, [(idx.cuda(), bad.cuda().to(dtype))])
        assert sdm.device_status() == sdm.SDM_DEV_BAD_INDEX
        assert torch.isfinite(want).all() and torch.equal(got, want)


@pytest.mark.parametrize("tokens", (9, 5000))
@pytest.mark.parametrize("hd,width", [(64, 7), (72, 40), (200, 33), (264, 5), (1000, 9), (37, 12)])
@pytest.mark.parametrize("format", ("int8", "fp8", "int4", "bf16", "f32"))
def test_gradients(tokens, hd, width, format):
    idx, out, gen = _entries(tokens, width, hd * tokens)
    dout = torch.randn((tokens, hd), generator=gen)
    bank = _bank(hd, format)
    fine, = quant.gather_dw(bank, [(idx.cuda(), dout.cuda())])
    assert (fine.cpu()[out] == 0).all() and torch.isfinite(fine).all()
    dout[:, 3] = torch.tensor([INF, NAN, -INF])[torch.arange(tokens) % 3]
    dout[2], dout[3] = NAN, INF
    for dtype in (torch.float32, torch.bfloat16):
        got, = quant.gather_dw(bank, [(idx.cuda(), dout.cuda())], dtype=dtype)
        assert (got.cpu()[out] == 0).all()
        assert not torch.isfinite(got.cpu()[~out]).any()  # a non-finite column meets every other row
    assert sdm.device_status() == sdm.SDM_DEV_BAD_INDEX
