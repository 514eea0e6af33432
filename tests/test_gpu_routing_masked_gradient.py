"""Gradients that belong to masked places change nothing, whatever they are: a weight that is 0 for any logit of
-inf or NaN has no gradient, so an infinity or NaN in its dw (a row that was never written, say) stays out of
the sums. Bits are the same as with dw = 0 there."""

from __future__ import annotations

import pytest
import torch

from decode_state_gb300 import routing, sdm

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ("softmax", "sigmoid"))
@pytest.mark.parametrize("renorm", (True, False))
@pytest.mark.parametrize("n,k", [(12, 6), (200, 40), (1000, 8), (1500, 64), (5000, 40), (20000, 100)])
@pytest.mark.parametrize("masked", (float("-inf"), float("nan")))
def test_masked_places(kind, renorm, n, k, masked):
    gen = torch.Generator().manual_seed(n + k)
    x = torch.randn((6, n), generator=gen)
    idx = torch.stack([torch.randperm(n, generator=gen)[:k] for _ in range(6)])
    dw = torch.randn((6, k), generator=gen)
    bad = dw.clone()
    for t in range(5):  # none to all of the chosen ones
        places = torch.randperm(k, generator=gen)[:t * k // 4]
        x[t, idx[t, places]] = masked
        dw[t, places] = 0.0
        bad[t, places] = torch.tensor([float("nan"), float("inf"), -float("inf")])[torch.arange(len(places)) % 3]
    kw = dict(score=kind, renorm=renorm)
    want = routing.route_backward(x.cuda(), idx.cuda(), dw.cuda(), **kw)
    got = routing.route_backward(x.cuda(), idx.cuda(), bad.cuda(), **kw)
    assert torch.isfinite(want).all() and torch.equal(got, want)
    assert (got.cpu()[x.isnan() | (x == -float("inf"))] == 0).all()


def test_indices_outside_the_row():
    """They are skipped with their dw."""
    x = torch.randn((2, 50), generator=torch.Generator().manual_seed(0)).cuda()
    idx = torch.tensor([[4, 50, 7], [-1, 2, 3]], device="cuda")
    dw = torch.tensor([[1.0, float("nan"), 2.0], [float("inf"), 3.0, -1.0]], device="cuda")
    sdm.device_status()
    for kind in ("softmax", "sigmoid"):
        for renorm in (True, False):
            d = routing.route_backward(x, idx, dw, score=kind, renorm=renorm)
            assert sdm.device_status() == sdm.SDM_DEV_BAD_INDEX
            want = routing.route_backward(x, idx, dw.nan_to_num(0.0, 0.0, 0.0), score=kind, renorm=renorm)
            assert sdm.device_status() == sdm.SDM_DEV_BAD_INDEX
            assert torch.isfinite(d).all() and torch.equal(d, want)
