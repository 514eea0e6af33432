"""The gradient of entries that fill up: where fewer than k entries are live, those of groups that do not stay and
those that a bias of -inf switches off fill up with weight 0, whatever their logits. They have no gradient of
their own and no part in the sums of the others.

The reference is central differences of the 64-bit forward definition, summed with dw by entry, at logits
whose choice does not change within the step h = 1e-5: truncation of order h^2 and rounding of order
2^-52 / h, together below 1e-9 for weights of order 1; the kernel is within 128 eps (8e-6) of magnitudes of
order 1 to 8, as in the tests without filled places. Tolerance: 1e-4.
"""

from __future__ import annotations

import numpy as np
import pytest
import quant_reference as ref
import torch

from decode_state_gb300 import quant, routing
from decode_state_gb300.state import RoutedLayerState

pytestmark = pytest.mark.gpu

INF = float("inf")
H = 1e-5


def _differences(x, by_entry, columns, **kw):
    """d loss / d logits of the 64-bit forward, loss = sum over the chosen of weight * by_entry[its index]."""
    kw = dict(kw)
    k, kind = kw.pop("k"), kw.pop("kind")

    def loss(y):
        idx, w = ref.route(y, k, kind, **kw)
        live = w != 0
        return (w * np.where(live, np.take_along_axis(by_entry, idx, 1), 0)).sum(1), np.sort(np.where(live, idx, -1), 1)

    _, chosen = loss(x)
    d = np.zeros((len(x), len(columns)))
    for i, j in enumerate(columns):
        e = np.zeros_like(x)
        e[:, j] = H
        (up, a), (down, b) = loss(x + e), loss(x - e)
        assert np.array_equal(a, chosen) and np.array_equal(b, chosen)
        d[:, i] = (up - down) / (2 * H)
    return d


CASES = [  # n, k, groups, top_groups, entries that a bias switches off
    (64, 16, 8, 1, 0), (32, 20, 4, 2, 0), (32, 20, 4, 2, 3), (40, 30, 1, 1, 25), (256, 40, 8, 1, 0), (256, 60, 8, 2, 30), (60, 12, 30, 3, 0),
    (1000, 64, 20, 1, 0), (2048, 100, 32, 1, 5), (1500, 200, 1, 1, 1400)]


def _case(n, k, groups, top_groups, off, kind, seed):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((3, n), generator=gen)
    x[1, torch.randperm(n, generator=gen)[:n // 4]] = -INF  # masked logits among them
    b = None
    if off:
        b = torch.rand(n, generator=gen) / 8
        b[torch.randperm(n, generator=gen)[:off]] = -INF
    by_entry = torch.randn((3, n), generator=gen)
    return x, b, by_entry, dict(groups=groups, top_groups=top_groups)


def _columns(n, idx):
    """All of a short row; of a long one the chosen entries, filled ones among them, and some others."""
    return np.arange(n) if n <= 64 else np.unique(np.concatenate([idx[:, ::7].ravel(), np.arange(0, n, n // 23)]))


@pytest.mark.parametrize("kind", ("softmax", "sigmoid"))
@pytest.mark.parametrize("renorm", (True, False))
@pytest.mark.parametrize("group_top", (1, 2))
@pytest.mark.parametrize("n,k,groups,top_groups,off", CASES)
def test_against_differences_of_the_forward(kind, renorm, group_top, n, k, groups, top_groups, off):
    x, b, by_entry, kw = _case(n, k, groups, top_groups, off, kind, n + k)
    kw.update(group_top=group_top, renorm=renorm, scale=1.5)
    idx, w = routing.route(x.cuda(), k, score=kind, bias=None if b is None else b.cuda(), idx_dtype=torch.int64, **kw)
    at = idx.cpu()
    assert (w == 0).any()  # some places are filled
    dw = by_entry.gather(1, at)
    d = routing.route_backward(x.cuda(), idx, dw.cuda(), score=kind, renorm=renorm, scale=1.5, w=w).cpu().double().numpy()
    cols = _columns(n, at.numpy())
    want = _differences(x.double().numpy(), by_entry.double().numpy(), cols, k=k, kind=kind,
                        bias=None if b is None else b.numpy(), **kw)
    assert np.abs(d[:, cols] - want).max() <= 1e-4
    # what fills up may have any dw
    dw[(w == 0).cpu()] = float("nan")
    again = routing.route_backward(x.cuda(), idx, dw.cuda(), score=kind, renorm=renorm, scale=1.5, w=w).cpu().double().numpy()
    assert np.array_equal(again, d)


@pytest.mark.parametrize("kind", ("softmax", "sigmoid"))
@pytest.mark.parametrize("renorm", (True, False))
@pytest.mark.parametrize("n,k", [(40, 8), (1000, 33), (3000, 40), (20000, 64)])
def test_weights_change_nothing_where_none_fills_up(kind, renorm, n, k):
    gen = torch.Generator().manual_seed(n)
    x = torch.randn((4, n), generator=gen)
    x[1, k // 2:] = -INF
    x[2] = -INF
    x = x.cuda()
    base = torch.arange(4, device="cuda", dtype=torch.int32) * n
    idx, w = routing.route(x, k, score=kind, renorm=renorm, base=base)
    dw = torch.randn((4, k), generator=gen).cuda()
    kw = dict(score=kind, renorm=renorm, base=base)
    assert torch.equal(routing.route_backward(x, idx, dw, w=w, **kw), routing.route_backward(x, idx, dw, **kw))


@pytest.mark.parametrize("kind", ("softmax", "sigmoid"))
@pytest.mark.parametrize("renorm", (True, False))
@pytest.mark.parametrize("router", ("groups", "bias"))
@pytest.mark.parametrize("given", (True, False))
def test_reading_of_the_state(kind, renorm, router, given):
    """RoutedLayerState: the readings' gradient through read_backward, with the weights of the reading or without."""
    streams, slots, hd, reads = 3, 48, 32, 20
    gen = torch.Generator().manual_seed(5)
    rows = torch.randn((streams * slots, hd), generator=gen)
    kw = dict(groups=6, top_groups=2) if router == "groups" else {}
    b = None
    if router == "bias":
        b = torch.rand(slots, generator=gen) / 8
        b[torch.randperm(slots, generator=gen)[:36]] = -INF
    bank = quant.QuantBank.from_rows(rows.cuda(), group=32)
    s = RoutedLayerState(bank, streams, writes=4, reads=reads, score=kind, renorm=renorm, scale=1.5,
                         **({} if b is None else {"bias": b.cuda()}), **kw)
    q = torch.randn((streams, slots), generator=gen)
    out, idx, w = s.read(q.cuda())
    assert (w == 0).any()
    dout = torch.randn((streams, hd), generator=gen) / 4
    d = (s.read_backward(q.cuda(), idx, dout.cuda(), w) if given else s.read_backward(q.cuda(), idx, dout.cuda())).cpu().double().numpy()
    held = s.rows(torch.float32).cpu().double().view(streams, slots, hd)
    by_entry = (held * dout.double()[:, None]).sum(2).numpy()
    want = _differences(q.double().numpy(), by_entry, np.arange(slots), k=reads, kind=kind, renorm=renorm, scale=1.5,
                        bias=None if b is None else b.numpy(), **kw)
    assert np.abs(d - want).max() <= 1e-4
