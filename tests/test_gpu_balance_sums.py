"""The balance loss of calls with thousands of rows a team, whose parts are nearly alike: their sum is as good as they are.

Tolerance. The logits lie within 2^-7 of each other, so a share is off by 4 steps of 2^-24 for its exponential, as many for the
sum of the row's (of which the additions, up to 16 in a lane and 10 joins, take 13 at half a step each), 2 for the reciprocal
and 1 each for the two products: 24. A team's sum carries what it loses and adds 2, the part before it 1, the team's
float32 sum 1. PARTS = 32 of what train_reference.balance says that one step of every share moves the loss by."""

from __future__ import annotations

import pytest
import torch

import train_reference as ref
from decode_state_gb300 import routing

pytestmark = pytest.mark.gpu

PARTS = 32.0


@pytest.mark.parametrize("n,tokens", ((32, 100_000_000), (256, 9_000_000), (600, 4_000_000)))
@pytest.mark.parametrize("score", ("softmax", "sigmoid"))
def test_many_rows_that_are_nearly_alike(n, tokens, score):
    x = torch.zeros((tokens, n), dtype=torch.bfloat16, device="cuda")
    idx = torch.arange(tokens, device="cuda", dtype=torch.int32).remainder_(n)
    idx[::10] = 0
    want = torch.bincount(idx, minlength=n)[None].cpu()
    for first in (2.0 ** -7, 2.0 ** -9, 2.0 ** -10):
        x[:, 0] = first
        # one row stands for all: the loss is n / C <c, p>
        l64, _, moved, _ = ref.balance(x[:1].cpu(), want, score=score)
        for gradient in (False, True):
            loss, counts, *_ = routing.balance(x, idx[:, None], score=score, gradient=gradient)
            assert torch.equal(counts.cpu().long(), want)
            ref.close(loss, l64, moved, f"loss, {first}", PARTS)
