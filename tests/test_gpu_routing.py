"""Routing on the GPU, forward and backward, against plain implementations in 64 bits.

Tolerances, fixed before the first run:
  choice     without a bias: exactly the 64-bit choice, since logits lie on a grid of 2^-7 within +-8,
             where distinct scores differ by far more than a float32 rounding. With a bias the
             64-bit ranks of what was chosen may be below those of what was left out, or out of
             order, by 8 eps (two roundings of a rank of at most 2) only.
  weights    64 eps of the value: exp to 2 ulp of an argument of at most 16 that is rounded once
             (16 eps absolute), a sum of positive terms, a division, a product
  gradient   128 eps of the magnitudes that it is made of, and one rounding to bfloat16 (2^-8)
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


def _logits(t, n, dtype, seed, masked=0.0):
    """On a grid of 2^-7 within +-8 in float32 (bf16 rounds to a coarser one), many equal."""
    gen = torch.Generator().manual_seed(seed)
    x = (torch.randn((t, n), generator=gen) * 2).clamp_(-8, 8)
    x = (x * 128).round() / 128
    if masked:
        x[torch.rand((t, n), generator=gen) < masked] = -float("inf")
    return x.to(dtype)


def _bias(n, seed):
    return torch.rand(n, generator=torch.Generator().manual_seed(seed)) * 0.5 - 0.25


def _check_weights(w, idx, x, kind, renorm, scale, live):
    want = np.take_along_axis(ref.scores(x, kind), idx, 1) * live
    if renorm:
        total = want.sum(1, keepdims=True)
        want = want / np.where(total > 0, total, 1)
    want = want * scale
    err = np.abs(w - want)
    assert (err <= 64 * EPS * want + 1e-37).all(), err.max()


SIZES = [(1, 1, 1), (1, 5, 5), (3, 8, 2), (70, 33, 7), (64, 256, 8), (37, 250, 32), (9, 513, 31), (5, 1024, 32), (5, 1000, 33),
         (20, 64, 64), (3, 1025, 8), (4, 4099, 64), (3, 5000, 256), (2, 16384, 64), (2, 65536, 33), (3000, 40, 3)]


@pytest.mark.parametrize("kind", ("softmax", "sigmoid"))
@pytest.mark.parametrize("dtype", (torch.bfloat16, torch.float32))
@pytest.mark.parametrize("t,n,k", SIZES)
def test_choice_without_bias(kind, dtype, t, n, k):
    x = _logits(t, n, dtype, n, masked=0.2 if n % 2 else 0.0)
    renorm, scale, it = bool(t % 2), 1.0 if n % 3 else 2.5, torch.int64 if k % 2 else torch.int32
    idx, w = routing.route(x.cuda(), k, score=kind, renorm=renorm, scale=scale, idx_dtype=it)
    assert idx.dtype == it and idx.shape == w.shape == (t, k)
    xn, idx, w = x.float().numpy(), idx.cpu().numpy().astype(np.int64), w.cpu().double().numpy()
    want, _ = ref.route(xn, k, kind)
    assert np.array_equal(idx, want)
    live = np.take_along_axis(xn, idx, 1) > -np.inf
    assert (w[~live] == 0).all()
    _check_weights(w, idx, xn, kind, renorm, scale, live)


GROUPED = [(64, 256, 8, 8, 4), (9, 96, 6, 4, 1), (33, 250, 10, 5, 2), (6, 60, 12, 30, 7), (4, 1024, 32, 256, 13), (5, 999, 40, 27, 5),
           (3, 2048, 64, 16, 3), (2, 16384, 100, 128, 9), (7, 24, 3, 24, 5), (5, 32, 20, 4, 2)]


@pytest.mark.parametrize("kind", ("softmax", "sigmoid"))
@pytest.mark.parametrize("group_top", (1, 2))
@pytest.mark.parametrize("t,n,k,groups,top_groups", GROUPED)
def test_groups_without_bias(kind, group_top, t, n, k, groups, top_groups):
    """A sum of two scores may tie within a rounding where the 64-bit sums differ, so the groups are
    judged with the tolerance and the entries within the groups that stayed exactly."""
    x = _logits(t, n, torch.float32, n + groups, masked=0.1 if k % 2 else 0.0)
    idx, w = routing.route(x.cuda(), k, score=kind, groups=groups, top_groups=top_groups, group_top=group_top)
    xn, idx, w = x.numpy(), idx.cpu().numpy().astype(np.int64), w.cpu().double().numpy()
    _check_grouped(xn, idx, w, kind, None, groups, top_groups, group_top)


def _check_grouped(xn, idx, w, kind, bias, groups, top_groups, group_top):
    t, n = xn.shape
    r = ref.ranks(xn, kind, bias)
    judged = ref.scores(xn, kind) if bias is None and kind == "softmax" and group_top == 2 else r
    judged = np.where(r == -np.inf, -np.inf, judged).reshape(t, groups, -1)
    best = -np.sort(-judged, axis=2)[..., :group_top]
    score = np.where(best[..., 0] == -np.inf, -np.inf, np.where(best == -np.inf, 0, best).sum(2))
    tol = 8 * EPS * (1 if bias is not None else np.maximum(np.abs(np.where(score == -np.inf, 0, score)).max(), 1e-30))
    per = n // groups
    for i in range(t):
        # the sets of groups that may stay: those clearly better than the top_groups-th, and some of those near it
        edge = np.sort(score[i])[::-1][top_groups - 1]
        near = np.abs(score[i] - edge) <= tol if edge > -np.inf else score[i] == edge
        if near.sum() == 1 or (score[i] > edge).sum() + near.sum() == top_groups or len(set(score[i][near])) == 1:
            order = np.argsort(-score[i], kind="stable")[:top_groups]
        else:  # a near tie: believe the kernel about which of the near ones stayed
            clear = np.flatnonzero((score[i] > edge) & ~near)
            used = [g for g in np.unique(idx[i][w[i] > 0] // per) if near[g]]
            order = np.concatenate([clear, np.array(used, int)])
            assert len(order) <= top_groups
        keep = np.isin(np.arange(n) // per, order)
        _check_order(np.where(keep, r[i], -np.inf), idx[i], w[i], exact=bias is None)
    live = w > 0
    _check_weights(w, idx, xn, kind, True, 1.0, live)


def _check_order(r, idx, w, exact):
    """idx is a best-first choice by the ranks r, exactly or within 8 eps."""
    k = len(idx)
    assert len(set(idx)) == k
    want = np.argsort(-r, kind="stable")[:k]
    if exact:
        assert np.array_equal(idx, want)
        return
    live = np.isfinite(r[idx])
    assert live.sum() == min(k, np.isfinite(r).sum()) and not (np.diff(live.astype(int)) > 0).any()
    got = r[idx][live]
    assert (np.diff(got) <= 8 * EPS).all()
    rest = np.delete(r, idx)
    if len(got) and np.isfinite(rest).any():
        assert rest.max() <= got.min() + 8 * EPS
    assert (w[~live] == 0).all()
    assert (np.diff(idx[~live]) > 0).all()


@pytest.mark.parametrize("kind", ("softmax", "sigmoid"))
@pytest.mark.parametrize("t,n,k,groups,top_groups", GROUPED)
def test_choice_with_bias(kind, t, n, k, groups, top_groups):
    x, b = _logits(t, n, torch.bfloat16, n, masked=0.15 if n % 2 else 0.0), _bias(n, t)
    b[n // 2] = -float("inf")  # an entry that is switched off
    for grouped in (False, True):
        for top in (1, 2):
            kw = dict(groups=groups, top_groups=top_groups, group_top=top) if grouped else {}
            idx, w = routing.route(x.cuda(), k, score=kind, bias=b.cuda(), **kw)
            xn, idx, w = x.float().numpy(), idx.cpu().numpy().astype(np.int64), w.cpu().double().numpy()
            if grouped:
                _check_grouped(xn, idx, w, kind, b.numpy(), groups, top_groups, top)
            else:
                r = ref.ranks(xn, kind, b.numpy())
                for i in range(t):
                    _check_order(r[i], idx[i], w[i], exact=False)
                _check_weights(w, idx, xn, kind, True, 1.0, np.isfinite(np.take_along_axis(r, idx, 1)))


@pytest.mark.parametrize("kind", ("softmax", "sigmoid"))
@pytest.mark.parametrize("n,k", [(40, 8), (700, 20), (3000, 70), (20000, 200)])
def test_masked_and_extreme_rows(kind, n, k):
    """Rows that are masked throughout, have fewer live entries than k, are all equal, hold NaN,
    infinities, the lowest float, or signed zeros."""
    x = torch.full((9, n), -float("inf"))
    x[1, 5] = 1.0
    x[1, n - 1] = 2.0
    x[2] = 0.25
    x[3] = float("nan")
    x[4, ::2] = torch.finfo(torch.float32).min
    x[5, 3], x[5, 9], x[5, 11] = float("inf"), float("inf"), 7.0
    x[6, :k] = torch.arange(k) * -0.01
    x[7, ::2], x[7, 1::2] = 0.0, -0.0
    x[8] = -200.0
    x[8, n // 2] = -100.0
    for renorm in (True, False):
        idx, w = routing.route(x.cuda(), k, score=kind, renorm=renorm)
        idx, w = idx.cpu().numpy().astype(np.int64), w.cpu().double().numpy()
        want, ww = ref.route(x.numpy(), k, kind, renorm=renorm)
        # the scores are float32: sigmoid(-100) is 0 there, and the last row's entries are all alike
        for i in [0, 1, 2, 3, 4, 5, 6, 7] if kind == "sigmoid" else range(9):
            assert np.array_equal(idx[i], want[i]), i
            assert np.allclose(w[i], ww[i], rtol=64 * EPS, atol=1e-37), i
        assert (w[0] == 0).all() and (w[3] == 0).all()
        assert np.array_equal(idx[0], np.arange(k)) and np.array_equal(idx[2], np.arange(k))


def test_strides_base_and_streams():
    """Logits as a slice of a wider projection, indices offset to each stream's slots, a stream of its own."""
    wide = _logits(50, 700, torch.bfloat16, 1).cuda()
    for lo, n in ((0, 256), (3, 300), (256, 256), (8, 600)):
        x = wide[:, lo:lo + n]
        base = (torch.arange(50, device="cuda") * 1000).to(torch.int64)
        want, ww = routing.route(x.contiguous(), 16, idx_dtype=torch.int64)
        idx, w = routing.route(x, 16, base=base, idx_dtype=torch.int64)
        assert torch.equal(idx, want + base[:, None]) and torch.equal(w, ww)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        again, w2 = routing.route(x, 16, base=base, idx_dtype=torch.int64, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(again, idx) and torch.equal(w2, w)
        dw = torch.randn(50, 16, device="cuda")
        for score in ("softmax", "sigmoid"):
            for renorm in (True, False):
                kw = dict(score=score, renorm=renorm)
                plain = routing.route_backward(x.contiguous(), want, dw, **kw)
                out = torch.full((50, n + 5), 7.0, dtype=torch.bfloat16, device="cuda")
                routing.route_backward(x, idx, dw, base=base, out=out[:, 2:2 + n], **kw)
                assert torch.equal(out[:, 2:2 + n], plain)
                assert (out[:, :2] == 7).all() and (out[:, 2 + n:] == 7).all()


def test_bad_indices_are_skipped_and_flagged():
    x = _logits(2, 50, torch.float32, 3).cuda()
    idx = torch.tensor([[4, 50, 7], [-1, 2, 3]], device="cuda")
    for renorm in (True, False):
        d = routing.route_backward(x, idx, torch.ones(2, 3, device="cuda"), score="sigmoid", renorm=renorm)
        assert sdm.device_status() == sdm.SDM_DEV_BAD_INDEX
        zero = d == 0
        assert zero.sum().item() >= 96 and torch.isfinite(d).all()


@pytest.mark.parametrize("kind", ("softmax", "sigmoid"))
@pytest.mark.parametrize("renorm", (True, False))
@pytest.mark.parametrize("dtype", (torch.bfloat16, torch.float32))
@pytest.mark.parametrize("t,n,k", [(1, 1, 1), (3, 7, 7), (70, 33, 6), (64, 256, 8), (9, 1023, 40), (5, 1025, 33), (4, 4099, 64),
                                   (2, 20001, 256), (1, 65536, 64), (2500, 40, 4)])
def test_gradient(kind, renorm, dtype, t, n, k):
    x = _logits(t, n, dtype, n + 1, masked=0.1 if n > 8 else 0.0)
    gen = torch.Generator().manual_seed(t)
    dw = torch.randn((t, k), generator=gen)
    idx = torch.stack([torch.randperm(n, generator=gen)[:k] for _ in range(t)])
    d = routing.route_backward(x.cuda(), idx.cuda(), dw.cuda(), score=kind, renorm=renorm, scale=1.5)
    want, size = ref.route_backward(x.float().numpy(), idx.numpy(), dw.numpy(), kind, renorm, 1.5)
    assert d.dtype == dtype
    tol = 128 * EPS * size + 1e-37 + (2.0 ** -8 * np.abs(want) if dtype == torch.bfloat16 else 0)
    err = np.abs(d.cpu().double().numpy() - want)
    assert (err <= tol).all(), (err - tol).max()
    assert (d.cpu().float().numpy()[x.float().numpy() == -np.inf] == 0).all()


@pytest.mark.parametrize("kind", ("softmax", "sigmoid"))
@pytest.mark.parametrize("renorm", (True, False))
def test_gradient_against_differences(kind, renorm):
    """Central differences of the 64-bit weights: truncation of order h^2, rounding of order 2^-52 / h."""
    t, n, k, h = 3, 40, 5, 1e-4
    x = _logits(t, n, torch.float32, 2)
    idx, _ = routing.route(x.cuda(), k, score=kind, renorm=renorm, idx_dtype=torch.int64)
    dw = torch.randn((t, k), generator=torch.Generator().manual_seed(0))
    d = routing.route_backward(x.cuda(), idx, dw.cuda(), score=kind, renorm=renorm, scale=2.0).cpu().double().numpy()
    xn, at = x.double().numpy(), idx.cpu().numpy()
    for j in range(n):
        e = np.zeros_like(xn)
        e[:, j] = h
        diff = (ref.weights_of(xn + e, at, kind, renorm, 2.0) - ref.weights_of(xn - e, at, kind, renorm, 2.0)) / (2 * h)
        assert np.abs((diff * dw.double().numpy()).sum(1) - d[:, j]).max() <= 1e-5


def test_many_tokens_and_nothing():
    x = _logits(1, 16, torch.float32, 5).cuda()
    many = x.expand(200001, 16).contiguous()
    idx, w = routing.route(many, 2)
    assert (idx == idx[0]).all() and (w == w[0]).all()
    d = routing.route_backward(many, idx, torch.ones_like(w) * torch.tensor([1.0, 0.0], device="cuda"))
    assert (d == d[0]).all()
    none = x[:0]
    idx, w = routing.route(none, 2)
    assert idx.shape == (0, 2) and routing.route_backward(none, idx, w).shape == (0, 16)
