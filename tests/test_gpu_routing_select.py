"""The choice of many of few: k from 1 to 200 of rows up to 1100 entries, where rows hold ties, few live
entries, values of any size, and groups of which few stay.

Indices are exact where ranks are the logits (softmax) or are compared as the float32 scores themselves:
ties go to the lower index. Weights are within 16 eps of the 64-bit ones, plus (k + 8) eps for the sum.
"""

from __future__ import annotations

import numpy as np
import pytest
import quant_reference as ref
import torch
from quant_reference import EPS

from decode_state_gb300 import routing, sdm

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status():
    sdm.device_status()
    yield
    assert sdm.device_status() == 0


def _rows(n, dtype, seed):
    """Rows of all kinds: spread, in steps of a quarter, on two values, nearly all masked, all alike, of every
    exponent, one far above the others, with both infinities and NaN, ascending and descending."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((10, n), generator=gen)
    x[1] = (x[1] * 4).round() / 4
    x[2] = (x[2] > 0.3).float()
    x[3, torch.rand(n, generator=gen) < 0.9] = -float("inf")
    x[4] = 0.5
    x[5] = x[5].sign() * torch.exp2(240 * torch.rand(n, generator=gen) - 120)
    x[6, n // 2] = 1e30
    x[7, 0], x[7, n // 3], x[7, n - 1] = float("nan"), float("inf"), -float("inf")
    x[8] = torch.arange(n) / 64
    x[9] = -torch.arange(n) / 64
    return x.to(dtype)


@pytest.mark.parametrize("dtype", (torch.bfloat16, torch.float32))
@pytest.mark.parametrize("n", (33, 64, 97, 200, 256, 500, 1000, 1024, 1100))
@pytest.mark.parametrize("k", (1, 31, 33, 48, 64, 65, 200))
def test_softmax_choice(dtype, n, k):
    if k > n:
        k = n
    x = _rows(n, dtype, n + k)
    idx, w = routing.route(x.cuda(), k)
    xn = x.double().numpy()
    r = np.where(np.isnan(xn), -np.inf, xn)
    want = np.argsort(-r, axis=1, kind="stable")[:, :k]
    assert np.array_equal(idx.cpu().numpy(), want)
    s = np.take_along_axis(ref.scores(x.float().numpy(), "softmax"), want, 1)
    s = s / s.sum(1, keepdims=True)
    # an exponential of a difference d has its rounding, |d| eps, in it; below 1e-30 it is as good as nothing
    top = r.max(axis=1, keepdims=True)
    d = np.where(s > 1e-30, np.abs(np.take_along_axis(r, want, 1) - np.where(np.isinf(top), 0, top)), 0)
    assert (np.abs(w.cpu().double().numpy() - s) <= (16 + k + 8 + 2 * d) * EPS * s + 1e-30).all()


@pytest.mark.parametrize("n", (64, 200, 512, 1000))
@pytest.mark.parametrize("k", (8, 40, 64))
def test_sigmoid_choice_and_scores(n, k):
    """Neither renormalised nor scaled, the weights are the float32 scores, best first, and they are the k
    largest of all scores: those of a row of n entries with k = n, in two halves."""
    x = _rows(n, torch.float32, n * k).cuda()
    idx, w = routing.route(x, k, score="sigmoid", renorm=False)
    every = torch.zeros_like(x)
    for a in range(0, n, 50):  # scores as float32 of all entries, 50 at a time
        part = x[:, a:a + 50].contiguous()
        i, s = routing.route(part, part.shape[1], score="sigmoid", renorm=False)
        every[:, a:a + 50].scatter_(1, i.long(), s)
    live = ~x.isnan() & (x != -float("inf"))
    rank = torch.where(live, every, -1.0)
    want = torch.argsort(-rank.cpu(), dim=1, stable=True)[:, :k].cuda()
    # equal scores go to the lower index, masked entries come last in index order
    assert torch.equal(idx.long(), want)
    assert torch.equal(w, every.gather(1, want))
    exact = ref.scores(x.cpu().numpy(), "sigmoid")
    assert (np.abs(every.cpu().double().numpy() - exact) <= 8 * EPS * exact + 1e-37).all()


@pytest.mark.parametrize("dtype", (torch.bfloat16, torch.float32))
@pytest.mark.parametrize("n,groups,top_groups", [(200, 2, 1), (200, 8, 1), (500, 5, 2), (1000, 8, 1), (1000, 20, 3), (1024, 32, 2),
                                                 (256, 8, 2), (96, 48, 20), (255, 85, 30)])
@pytest.mark.parametrize("k", (8, 25, 32, 60))
def test_few_groups_stay(dtype, n, groups, top_groups, k):
    """Ranks are the logits and groups are judged by their best one, so everything is exact."""
    k = min(k, n)
    x = _rows(n, dtype, n + groups)
    idx, w = routing.route(x.cuda(), k, groups=groups, top_groups=top_groups)
    xn = np.where(np.isnan(x.double().numpy()), -np.inf, x.double().numpy())
    r = ref.drop_groups(xn, xn, "softmax", None, groups, top_groups, 1)
    want = np.argsort(-r, axis=1, kind="stable")[:, :k]
    assert np.array_equal(idx.cpu().numpy(), want)
    assert ((w.cpu().numpy() == 0) | (np.take_along_axis(r, want, 1) > -np.inf)).all()
