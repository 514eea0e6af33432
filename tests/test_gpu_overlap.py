"""Memory side by side and in place: what the calls take and what they refuse."""

from __future__ import annotations

import pytest
import torch

from decode_state_gb300 import quant, routing, sdm

pytestmark = pytest.mark.gpu


def _randn(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).cuda()


@pytest.mark.parametrize("n,k", [(64, 8), (100, 64), (1500, 40)])
@pytest.mark.parametrize("renorm", (True, False))
def test_gradient_beside_its_logits(n, k, renorm):
    """Logits and their gradient as the two halves of a matrix, and in place, where the gradient of the first
    entries would be read as a logit of the last."""
    wide = _randn(50, 2 * n + 3)
    x, out = wide[:, :n], wide[:, n + 3:]
    idx, w = routing.route(x, k, renorm=renorm)
    dw = _randn(50, k, seed=1)
    want = routing.route_backward(x.contiguous(), idx, dw, renorm=renorm)
    assert torch.equal(routing.route_backward(x, idx, dw, renorm=renorm, out=out), want)
    y, out = wide[:, n + 3:], wide[:, :n]  # the other way about
    y.copy_(_randn(50, n, seed=2))
    idx, w = routing.route(y, k, renorm=renorm)
    want = routing.route_backward(y.contiguous(), idx, dw, renorm=renorm)
    assert torch.equal(routing.route_backward(y, idx, dw, renorm=renorm, out=out), want)
    for bad in (y, wide[:, n:2 * n], wide[:, 4:n + 4]):
        with pytest.raises(sdm.SDMError):
            routing.route_backward(y, idx, dw, renorm=renorm, out=bad)


def test_weights_between_rows():
    """One token's weights and slots in the gap behind its logits, a small array in the gap of a row."""
    wide = torch.zeros(4, 200, device="cuda")
    wide[:, :100] = _randn(4, 100)
    x = wide[:, :100]
    want, ww = routing.route(x.contiguous(), 8)
    w = wide.view(-1)[300:332].view(4, 8)
    idx, got = routing.route(x, 8, w=w)
    assert torch.equal(idx, want) and torch.equal(w, ww) and got is w
    for at in (290, 380, 0, 599):
        with pytest.raises(sdm.SDMError):
            routing.route(x, 8, w=wide.view(-1)[at:at + 32].view(4, 8))


def test_rows_beside_one_another_and_in_the_bank():
    wide = _randn(60, 96)
    bank = quant.QuantBank.from_rows(wide[:, :64], group=32)
    out = wide[:, 64:96]
    half = quant.QuantBank.from_rows(wide[:, :32], group=32)
    quant.dequantize_rows(half, dtype=torch.float32, out=out)
    assert torch.equal(out, quant.dequantize_rows(half, dtype=torch.float32))
    held = bank.codes.view(-1)[:60 * 64].view(torch.float32).view(15, 64)
    with pytest.raises(sdm.SDMError):
        quant.dequantize_rows(bank, torch.arange(15, device="cuda"), out=held)
    with pytest.raises(sdm.SDMError):
        quant.quantize_rows(bank, held, torch.arange(15, device="cuda"))


@pytest.mark.parametrize("hd", (64, 200))
def test_readings_in_the_place_of_v(hd):
    gen = torch.Generator().manual_seed(3)
    T, S, P = 5, 6, 40
    a = quant.QuantBank.from_rows(_randn(S * P, hd), group=64)
    b = quant.QuantBank.from_rows(_randn(S * P, hd), group=64)
    at = torch.stack([torch.stack([torch.randperm(P, generator=gen)[:8] + s * P for s in range(S)]) for _ in range(T)]).cuda()
    k, q, v = _randn(T, S, 8, seed=4) / 3, _randn(T, S, 8, seed=5), _randn(T, S, hd, seed=6)
    beta, g = torch.rand(T, S, generator=gen).cuda(), -torch.rand(T, S, 1, generator=gen).cuda()
    want = quant.decode_seq(a, at, k, v, beta, g, at, q, out_dtype=torch.float32)
    got = quant.decode_seq(b, at, k, v, beta, g, at, q, out=v)
    assert got is v and torch.equal(v, want) and torch.equal(a.codes, b.codes)


def test_readings_over_what_the_decode_reads():
    S, hd = 6, 64
    bank = quant.QuantBank.zeros(S * 20, hd, group=32, device="cuda")
    at = (torch.arange(S, device="cuda") * 20)[:, None] + torch.arange(8, device="cuda")
    k, q, v = _randn(S, 64, seed=4)[:, :8].contiguous(), _randn(S, 8, seed=5), _randn(S, hd, seed=6)
    beta, g = torch.ones(S, device="cuda"), torch.zeros(S, 1, device="cuda")
    for taken in (bank.codes, bank.scales, v):
        out = taken.view(torch.bfloat16).view(-1)[:S * hd].view(S, hd)
        with pytest.raises(sdm.SDMError):
            quant.decode_step(bank, at, k, v, beta, g, at, q, out=out)
    assert not bank.codes.any()
