"""Renormalised weights, and their gradient, where all chosen scores are tiny: their sum is subnormal or so
small that its reciprocal overflows, while the weights themselves are ordinary numbers.

Tolerance: a float32 score s has an error of half the least float (2^-150) more than its 20 eps (exp of an
argument of at most 104 that is rounded once is within 2 ulp of that, and equal arguments give equal scores);
a weight s / S * scale has the relative errors of s and S and 3 eps, so 2 * (20 eps + 2^-150 / s) + 3 eps.
Equal logits have equal scores, whose errors cancel but for the sum's roundings, k eps.
"""

from __future__ import annotations

import numpy as np
import pytest
import quant_reference as ref
import torch
from quant_reference import EPS

from decode_state_gb300 import routing

pytestmark = pytest.mark.gpu

SIZES = [(8, 1), (64, 8), (256, 8), (200, 40), (1000, 8), (1000, 60), (1100, 8), (5000, 100)]


def _tolerance(s, w, k):
    return np.abs(w) * (2 * (20 * EPS + 2.0 ** -150 / s) + (3 + k) * EPS)


def _sigmoid_rows(n, k, scale, gen):
    x = torch.full((4, n), -88.5)
    x[1] = -86.0 - 2.5 * torch.rand(n, generator=gen)
    x[2] = -60.0 - 28.0 * torch.rand(n, generator=gen)
    x[3] = -88.0
    idx, w = routing.route(x.cuda(), k, score="sigmoid", scale=scale, idx_dtype=torch.int64)
    return x, idx, w, np.take_along_axis(ref.scores(x.numpy(), "sigmoid"), idx.cpu().numpy(), 1)


@pytest.mark.parametrize("n,k", SIZES)
@pytest.mark.parametrize("scale", (1.0, 2.5, 100.0))
def test_sigmoid_weights(n, k, scale):
    _, _, w, s = _sigmoid_rows(n, k, scale, torch.Generator().manual_seed(n + k))
    want = s / s.sum(1, keepdims=True) * scale
    assert (np.abs(w.cpu().double().numpy() - want) <= _tolerance(s, want, k)).all()


@pytest.mark.parametrize("n,k", SIZES)
@pytest.mark.parametrize("scale", (1.0, 2.5, 100.0))
def test_sigmoid_gradient(n, k, scale):
    gen = torch.Generator().manual_seed(n + k)
    x, idx, _, s = _sigmoid_rows(n, k, scale, gen)
    at, xn = idx.cpu().numpy(), x.numpy()
    dw = torch.randn((4, k), generator=gen)
    d = routing.route_backward(x.cuda(), idx, dw.cuda(), score="sigmoid", scale=scale).cpu().double().numpy()
    grad, size = ref.route_backward(xn, at, dw.numpy(), "sigmoid", True, scale)
    rel = (2 * (20 * EPS + 2.0 ** -150 / s) + (8 + k) * EPS).max(1, keepdims=True)
    assert (np.abs(d - grad) <= 2 * rel * size).all()


@pytest.mark.parametrize("n,k", SIZES)
def test_biased_softmax_weights(n, k):
    """The bias chooses entries whose exponentials are subnormal; one entry far above them is not chosen."""
    gen = torch.Generator().manual_seed(n * k)
    x = torch.zeros((3, n))
    x[0, 1:] = -95.0
    x[1, 1:] = -89.0 - 10 * torch.rand(n - 1, generator=gen)
    x[2, 1:] = -87.4
    b = torch.ones(n)
    b[0] = -4.0
    for scale in (1.0, 2.5):
        idx, w = routing.route(x.cuda(), k, bias=b.cuda(), scale=scale)
        at = idx.cpu().numpy().astype(np.int64)
        assert (at > 0).all()
        s = np.take_along_axis(ref.scores(x.numpy(), "softmax"), at, 1)
        want = s / s.sum(1, keepdims=True) * scale
        assert (np.abs(w.cpu().double().numpy() - want) <= _tolerance(s, want, k)).all()


@pytest.mark.parametrize("n,k", [(64, 8), (1100, 8)])
def test_scores_of_zero_have_no_weight(n, k):
    x = torch.zeros((1, n))
    x[0, 1:] = -120.0
    b = torch.ones(n)
    b[0] = -4.0
    _, w = routing.route(x.cuda(), k, bias=b.cuda())
    assert (w == 0).all()
