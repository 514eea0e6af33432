"""The quotients that kernels form without a division, for every significand: all must have the bits of a
correctly rounded division, so everything is compared exactly."""

from __future__ import annotations

import math

import pytest
import torch

from decode_state_gb300 import quant, routing

pytestmark = pytest.mark.gpu

LEVELS = {"int8": 127.0, "fp8": 448.0, "int4": 7.0}


def _expected(x, y, level):
    """float32 on the CPU: the scales of groups (x, y) with x the larger, and y's value before rounding."""
    return x / level, y * (torch.full_like(x, level) / x)


def _check(x, share, fmt):
    """Rows of x and of the float next to share * x: `share` puts its code half way between two numbers, where
    an error in the last place of the factor turns the rounding."""
    level = LEVELS[fmt]
    y = (x.double() * share).float()
    rows = torch.stack([x, y], 1)
    bank = quant.QuantBank.from_rows(rows.cuda(), group=32, format=fmt)
    scale, value = _expected(x, y, level)
    assert torch.equal(bank.scales[:, 0].cpu(), scale)
    codes = bank.codes.cpu()
    if fmt == "int4":
        assert (codes[:, 0] & 15 == 7).all()
        assert torch.equal(codes[:, 0] >> 4, value.round().to(torch.uint8))
    elif fmt == "int8":
        assert (codes[:, 0] == 127).all()
        assert torch.equal(codes[:, 1], value.round().to(torch.uint8))
    else:
        assert (codes[:, 0] == 0x7e).all()
        assert torch.equal(codes[:, 1], value.to(torch.float8_e4m3fn).view(torch.uint8))


def _halves(n, fmt, seed):
    """Shares of the largest value that lie half way between two codes."""
    gen = torch.Generator().manual_seed(seed)
    if fmt == "fp8":  # between two neighbours of three bits behind the leading one
        e = torch.randint(-6, 8, (n,), generator=gen).double()
        return (1 + (torch.randint(0, 8, (n,), generator=gen).double() + 0.5) / 8) * torch.exp2(e) / LEVELS[fmt]
    return (torch.randint(0, int(LEVELS[fmt]), (n,), generator=gen).double() + 0.5) / LEVELS[fmt]


@pytest.mark.parametrize("fmt", sorted(LEVELS))
def test_scales_and_factors_of_every_significand(fmt):
    x = (torch.arange(1 << 23, dtype=torch.int32) + 0x3f800000).view(torch.float32)  # [1, 2)
    _check(x, _halves(len(x), fmt, 0), fmt)


@pytest.mark.parametrize("fmt", sorted(LEVELS))
def test_scales_and_factors_of_every_exponent(fmt):
    for e in list(range(-100, 128)):
        gen = torch.Generator().manual_seed(e + 200)
        s = torch.randint(0, 1 << 23, (512,), generator=gen, dtype=torch.int32)
        s[:2] = torch.tensor([0, (1 << 23) - 1], dtype=torch.int32)
        _check((s + ((e + 127) << 23)).view(torch.float32), _halves(512, fmt, e + 500), fmt)


def test_sigmoid_ranks_are_the_weights():
    """The scores that entries are ranked by and those that are returned come from different instructions and are
    the same floats: 1 + exp(-x) takes nearly every value of [1, 2], neighbours in the same row in any order."""
    y = 1 + torch.arange(1, (1 << 23) + 1, dtype=torch.float64) / (1 << 23)
    x = (-torch.log(y - 1)).float().view(-1, 256)
    gen = torch.Generator().manual_seed(0)
    order = torch.rand(x.shape, generator=gen).argsort(1)
    x = x.gather(1, order)
    ties = 0
    for part in x.split(8192):
        idx, w = routing.route(part.cuda(), 256, score="sigmoid", renorm=False)
        assert (w[:, 1:] <= w[:, :-1]).all()
        equal = w[:, 1:] == w[:, :-1]
        assert (~equal | (idx[:, 1:] > idx[:, :-1])).all()
        assert math.isclose(float(w.max()), 1 / (1 + math.exp(-float(part.max()))), rel_tol=1e-6)
        ties += int(equal.sum())
    assert ties > 0  # near 1 / 2 neighbours share a score
