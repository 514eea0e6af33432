"""The softmax sum of a block's rows: the same bits in every token of the same row, and the 64-bit weights.

The sum is read by every warp of a block and followed by other shared values without a barrier in between,
so a place that held both would change under a slow warp's reads.

Tolerance: 64 eps of the value (16 for the rounding of an exponential's argument of at most 16, the sum of at
most 128 positive terms a thread, whose roundings are far from all of one sign, a division and a product).
"""

from __future__ import annotations

import numpy as np
import pytest
import quant_reference as ref
import torch
from quant_reference import EPS

from decode_state_gb300 import routing

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,k,tokens", [(1100, 8, 20000), (1500, 64, 8192), (5000, 200, 4096), (20000, 8, 1024), (300, 100, 20000)])
@pytest.mark.parametrize("biased", (False, True))
def test_equal_rows_have_equal_weights(n, k, tokens, biased):
    gen = torch.Generator().manual_seed(n + k)
    x = (torch.randn((1, n), generator=gen) * 2).clamp_(-8, 8)
    b = torch.rand(n, generator=gen) if biased else None
    many = x.cuda().expand(tokens, n).contiguous()
    want, ww = ref.route(x.numpy(), k, "softmax", bias=None if b is None else b.numpy(), renorm=False)
    for _ in range(20):
        idx, w = routing.route(many, k, renorm=False, bias=None if b is None else b.cuda())
        assert torch.equal(idx, idx[:1].expand_as(idx)) and torch.equal(w, w[:1].expand_as(w))
    idx, w = idx[0].cpu().numpy().astype(np.int64), w[0].cpu().double().numpy()
    if b is None:
        assert np.array_equal(idx, want[0])
    own = ref.scores(x.numpy(), "softmax")[0, idx]  # of what was chosen: biased ranks may tie within a rounding
    assert (np.abs(w - own) <= 64 * EPS * own).all()
    assert len(set(idx) & set(want[0])) >= k - 2
