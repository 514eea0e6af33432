"""Rows with many infinite ranks: more equal ones than a block keeps candidates of, and all kinds of places
for them. Logits of +inf share a softmax evenly, and equal ranks go to the lower index.

Choices are exact; weights within 64 eps of the 64-bit ones (a sum of up to 65536 equal exponentials, which
are small integers and add up exactly, a division and a product).
"""

from __future__ import annotations

import numpy as np
import pytest
import quant_reference as ref
import torch
from quant_reference import EPS

from decode_state_gb300 import routing, sdm

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.fixture(autouse=True)
def _clean_status():
    sdm.device_status()
    yield
    assert sdm.device_status() == 0


def _rows(n, dtype, seed):
    """Rows with 5, 511, 512, 513 and 600 entries of +inf at random places, at the end, and everywhere."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((8, n), generator=gen)
    for i, m in enumerate((5, 511, 512, 513, 600)):
        x[i, torch.randperm(n, generator=gen)[:m]] = INF
    x[5, n - 600:] = INF
    x[6] = INF
    x[7] = -INF  # and a row with nothing else that is live
    x[7, torch.randperm(n, generator=gen)[:700]] = INF
    return x.to(dtype)


@pytest.mark.parametrize("n", (1100, 9000, 16384, 65536))
@pytest.mark.parametrize("k", (8, 64, 256))
@pytest.mark.parametrize("dtype", (torch.bfloat16, torch.float32))
def test_many_infinite_logits(n, k, dtype):
    x = _rows(n, dtype, n + k)
    for renorm in (True, False):
        idx, w = routing.route(x.cuda(), k, renorm=renorm)
        want, ww = ref.route(x.float().numpy(), k, "softmax", renorm=renorm)
        assert np.array_equal(idx.cpu().numpy(), want)
        assert (np.abs(w.cpu().double().numpy() - ww) <= 64 * EPS * ww).all()


@pytest.mark.parametrize("n", (1100, 9000, 65536))
@pytest.mark.parametrize("groups,top_groups", [(1, 1), (4, 2)])
@pytest.mark.parametrize("kind", ("softmax", "sigmoid"))
@pytest.mark.parametrize("k", (8, 70))
def test_many_infinite_biases(n, groups, top_groups, kind, k):
    """Entries that a bias of +inf forces on: more than 512 of them, also in the groups that stay."""
    gen = torch.Generator().manual_seed(n + k)
    x = torch.randn((3, n), generator=gen)
    for many in (600, n):
        b = torch.zeros(n)
        b[torch.randperm(n, generator=gen)[:many]] = INF
        kw = dict(groups=groups, top_groups=top_groups)
        idx, w = routing.route(x.cuda(), k, score=kind, bias=b.cuda(), **kw)
        want, ww = ref.route(x.numpy(), k, kind, bias=b.numpy(), **kw)
        assert np.array_equal(idx.cpu().numpy(), want)
        assert (np.abs(w.cpu().double().numpy() - ww) <= 64 * EPS * ww).all()


@pytest.mark.parametrize("n,k", [(1100, 8), (9000, 64), (65536, 200)])
@pytest.mark.parametrize("value", (-3.402823466e38, -1.0, 0.0, 3.402823466e38))
def test_many_equal_logits_below_few(n, k, value):
    """More than 512 equal last ranks of any size, the lowest and the largest float among them."""
    x = torch.full((3, n), -INF)
    x[0] = value
    x[1, n - 900:] = value
    x[2, ::2] = value
    if value < 3e38:
        x[:, n // 3], x[:, n - 2] = 3.402823466e38, INF
    idx, _ = routing.route(x.cuda(), k)
    want, _ = ref.route(x.numpy(), k, "softmax")
    assert np.array_equal(idx.cpu().numpy(), want)
