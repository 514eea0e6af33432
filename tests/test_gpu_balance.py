"""The balance loss, its counts and its gradient against a plain form in 64 bits, on every kernel path.

Tolerances. A share is an exponential over a sum. The exponential is off by 4 steps of 2^-24 and by 2.5 more for each unit of its
argument (a difference, a product and a constant are rounded), which is up to 60 here: 154. The sum's positive terms are
as far off as they, weighted by their size, so that those near the largest, with few units, decide; adding up to 128 of them a
thread and ten joins, the products and quotients that follow, with half a step each on average, take no more than the
remaining 46. So each share is off by at most PARTS = 200 steps of 2^-24, and the outputs by what that moves them by
(train_reference.balance), plus one rounding to their type."""

from __future__ import annotations

import pytest
import torch

import train_reference as ref
from decode_state_gb300 import routing, sdm

pytestmark = pytest.mark.gpu

PARTS = 200.0


def _inputs(tokens, n, k, dtype, seed=0, spread=2.0):
    gen = torch.Generator().manual_seed(seed)
    x = (torch.randn(tokens, n, generator=gen) * spread + torch.randn(n, generator=gen) * 0.5).to(dtype)
    idx = torch.rand(tokens, n, generator=gen).add_(x.float() * 0.1).topk(k, dim=1).indices
    return x, idx, gen


def _check(x, idx, *, score, w=None, base=None, offsets=None, scale=1.0, dloss=None, add=None, device=None, idx_dtype=torch.int32, **kw):
    """One call with the gradient and one without, both against the plain form; returns the gradient."""
    n = x.shape[1]
    to = lambda t, ty=None: None if t is None else t.to("cuda", ty)  # noqa: E731
    device = x.cuda() if device is None else device
    args = dict(score=score, w=to(w), base=to(base, idx_dtype), offsets=to(offsets, torch.int32), scale=scale)
    sdm.device_status()
    loss, counts, grad = routing.balance(device, to(idx, idx_dtype), gradient=True, dloss=to(dloss), add=to(add), **args, **kw)
    alone = routing.balance(device, to(idx, idx_dtype), **args)
    assert sdm.device_status() == 0
    assert len(alone) == 2 and torch.equal(alone[0], loss) and torch.equal(alone[1], counts)
    want = ref.count(idx, n, w=w, base=base, offsets=offsets)
    assert counts.dtype == torch.int32 and torch.equal(counts.cpu().long(), want)
    l64, g64, moved_l, moved_g = ref.balance(x, want, score=score, offsets=offsets, scale=scale, dloss=dloss, add=add)
    ref.close(loss, l64, moved_l, "loss", PARTS)
    if add is not None:
        moved_g = moved_g + ref.STEP * g64.abs() / PARTS  # one more sum
    ref.close(grad, g64, moved_g, "gradient", PARTS)
    return grad


SIZES = (1, 2, 7, 8, 9, 31, 32, 33, 64, 65, 100, 128, 130, 256, 257, 300, 512, 520, 1000, 1024, 1025, 2048, 2050, 4096, 4099, 8192, 8200,
         16384, 16385, 20000, 65536)


@pytest.mark.parametrize("n", SIZES)
@pytest.mark.parametrize("dtype", (torch.float32, torch.bfloat16))
@pytest.mark.parametrize("score", ("softmax", "sigmoid"))
def test_row_lengths(n, dtype, score):
    tokens = 67 if n <= 2048 else 9
    x, idx, _ = _inputs(tokens, n, min(n, 5), dtype, seed=n)
    _check(x, idx, score=score, scale=1.5)


@pytest.mark.parametrize("tokens", (1, 2, 3, 31, 32, 129, 5000, 70001))
@pytest.mark.parametrize("n,k", ((16, 4), (48, 48), (256, 8)))
def test_token_counts(tokens, n, k):
    x, idx, _ = _inputs(tokens, n, k, torch.bfloat16, seed=tokens)
    _check(x, idx, score="sigmoid", idx_dtype=torch.int64)


@pytest.mark.parametrize("n", (24, 64, 200, 1024, 1500, 6000, 17000))
@pytest.mark.parametrize("score", ("softmax", "sigmoid"))
def test_sequences(n, score):
    """Packed sequences, some empty, tokens before the first and behind the last; weights of 0; base; what comes for each
    loss; a gradient to add to."""
    tokens = 300
    x, idx, gen = _inputs(tokens, n, 6, torch.float32, seed=n)
    offsets = torch.tensor([4, 4, 5, 5, 5, 90, 91, 250, 250, 290], dtype=torch.int32)
    w = torch.rand(tokens, 6, generator=gen)
    w[torch.rand(tokens, 6, generator=gen) < 0.2] = 0
    w[5:90] = 0  # a sequence none of whose entries counts
    base = torch.randint(0, 1 << 20, (tokens,), generator=gen)
    dloss = torch.randn(9, generator=gen)
    add = torch.randn(tokens, n, generator=gen) * 1e-3
    grad = _check(x, idx + base[:, None], score=score, w=w, base=base, offsets=offsets, scale=0.7, dloss=dloss, add=add)
    outside = torch.cat([torch.arange(4), torch.arange(5, 90), torch.arange(290, tokens)])
    assert torch.equal(grad.cpu()[outside], add[outside])
    loss, counts, grad = routing.balance(x.cuda(), (idx + base[:, None]).cuda(), score=score, base=base.cuda(), offsets=offsets.cuda(),
                                         gradient=True)
    assert not grad[:4].any() and not grad[290:].any()


@pytest.mark.parametrize("sequences", (0, 1, 200, 5000))
def test_many_sequences(sequences):
    tokens, n = 2000, 40
    x, idx, gen = _inputs(tokens, n, 3, torch.bfloat16, seed=sequences)
    cuts = torch.randint(0, tokens + 1, (max(sequences - 1, 0),), generator=gen).sort().values
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64), cuts, torch.full((1,), tokens)])[:sequences + 1]
    _check(x, idx, score="softmax", offsets=offsets.to(torch.int32))


@pytest.mark.parametrize("n", (8, 20, 60, 100, 256, 700, 3000, 10000, 30000))
@pytest.mark.parametrize("dtype", (torch.float32, torch.bfloat16))
@pytest.mark.parametrize("score", ("softmax", "sigmoid"))
def test_masked_infinite_and_far_logits(n, dtype, score):
    x, idx, gen = _inputs(24, n, 4, dtype, seed=n)
    x[0] = -torch.inf
    x[1] = torch.nan
    x[2, : n // 2] = -torch.inf
    x[3, ::2] = torch.nan
    x[4, 1] = torch.inf
    x[5, [0, n - 1]] = torch.inf
    x[6] = torch.inf
    x[7] = -200.0  # sigmoid scores below the least float
    x[8] = -100.0 - torch.arange(n).to(dtype) % 7
    x[9] = -80.0
    x[10] = 60.0
    x[11] = -torch.finfo(dtype).max  # a mask of the type's lowest value
    x[12, 1:] = -torch.finfo(dtype).max
    x[13] = torch.finfo(dtype).max
    x[14] = 0.0
    x[15, 0] = 1e4
    x[16, 0], x[16, 1:] = 30.0, -30.0
    _check(x, idx, score=score)


@pytest.mark.parametrize("n", (40, 300, 900, 20000))
@pytest.mark.parametrize("offset", (3e4, -3e4, 1e7, -1e7, 3e10, -3e10, 2e38, -2e38))
def test_logits_far_from_zero(n, offset):
    """Rows whose logits differ by little and lie anywhere."""
    x, idx, gen = _inputs(9, n, 4, torch.float32, seed=n)
    steps = torch.randint(0, 6, (9, n), generator=gen).float() * max(1.0, abs(offset) * 2.0 ** -23)  # whole units in the last place
    _check(steps + offset, idx, score="softmax")


@pytest.mark.parametrize("n", (20, 300, 2000, 18000))
@pytest.mark.parametrize("offset", (-10.0, -25.0, -45.0, -70.0, -86.0))
def test_tiny_sigmoid_scores(n, offset):
    """Shares of scores far below one, some of them 0 in float32."""
    x, idx, gen = _inputs(14, n, 4, torch.float32, seed=n, spread=8.0)
    x, want = x + offset, ref.count(idx, n)
    loss, counts, grad = routing.balance(x.cuda(), idx.cuda(), score="sigmoid", gradient=True)
    l64, g64, moved_l, moved_g = ref.balance(x, want, score="sigmoid")
    ref.close(loss, l64, moved_l, "loss", PARTS)
    # a score below 2^-126 is 0 where the row's scores sum to 2^-30 or more: its share, up to 2^-96, is left out
    left_out = 2.0 ** -96 * n * (counts.cpu().double().max() + 1) / (14 * 56)
    ref.close(grad, g64, moved_g + left_out / PARTS, "gradient", PARTS)


def test_counts_far_from_even():
    """All choices on one entry, and on two; a loss of n for shares on one entry."""
    n, tokens = 64, 500
    x = torch.full((tokens, n), -torch.inf)
    x[:, 3] = 1.0
    idx = torch.full((tokens, 1), 3)
    loss, counts = routing.balance(x.cuda(), idx.cuda())
    assert float(loss) == n and int(counts[0, 3]) == tokens
    x = torch.zeros(tokens, n)
    loss, counts, grad = routing.balance(x.cuda(), idx.cuda(), gradient=True)
    assert float(loss) == 1.0
    _check(x, idx, score="softmax")


@pytest.mark.parametrize("score", ("softmax", "sigmoid"))
@pytest.mark.parametrize("n", (24, 300, 2100))
def test_gradient_against_differences(score, n):
    """Central differences of the plain loss, counts fixed, along random directions."""
    x, idx, gen = _inputs(12, n, 3, torch.float32, seed=n)
    offsets = torch.tensor([0, 5, 12], dtype=torch.int32)
    counts = ref.count(idx, n, offsets=offsets)
    _, _, grad = routing.balance(x.cuda(), idx.cuda(), score=score, offsets=offsets.cuda(), gradient=True)
    for _ in range(4):
        v = torch.randn(x.shape, generator=gen, dtype=torch.float64)
        h = 1e-5  # the second-order error is h^2, rounding 1e-16 / h
        up, down = (ref.balance(x.double() + d * v, counts, score=score, offsets=offsets)[0].sum() for d in (h, -h))
        slope, along = float((up - down) / (2 * h)), float((grad.cpu().double() * v).sum())
        assert abs(slope - along) <= 1e-5 * float((grad.cpu().double() * v).abs().sum()) + 1e-8


def _strided(x, pad, shift, dtype):
    wide = torch.full((len(x) * (x.shape[1] + pad) + shift + 8,), float("nan"), dtype=dtype, device="cuda")
    view = wide[shift:shift + len(x) * (x.shape[1] + pad)].view(len(x), -1)[:, :x.shape[1]]
    view.copy_(x)
    return wide, view


@pytest.mark.parametrize("n,pad,shift", ((256, 8, 0), (256, 0, 1), (100, 1, 0), (64, 3, 5), (1000, 24, 2), (5000, 1, 1), (17000, 8, 4)))
@pytest.mark.parametrize("dtype", (torch.float32, torch.bfloat16))
def test_strides_and_alignment(n, pad, shift, dtype):
    """Rows inside a wider matrix; what lies beside them stays."""
    x, idx, gen = _inputs(40, n, 4, dtype, seed=n + pad)
    _, view = _strided(x, pad, shift, dtype)
    wide, out = _strided(torch.zeros_like(x), pad, shift, dtype)
    add = (torch.randn(x.shape, generator=gen) * 1e-3).to(dtype)
    _, added = _strided(add, pad, shift, dtype)
    before = wide.clone()
    for given in (None, added):
        args = dict(device=view, out=out) if given is None else dict(device=view, out=out, add=add)
        _check(x, idx, score="softmax", **args)
    inside = torch.zeros(wide.shape, dtype=torch.bool, device="cuda")
    inside[shift:shift + 40 * (n + pad)].view(40, -1)[:, :n] = True
    assert torch.equal(wide.view(torch.int16 if dtype == torch.bfloat16 else torch.int32)[~inside],
                       before.view(torch.int16 if dtype == torch.bfloat16 else torch.int32)[~inside])
    want = routing.balance(view, idx.cuda(), gradient=True, add=added)[2]
    got = routing.balance(view, idx.cuda(), gradient=True, add=added, out=added)[2]  # in the place of what it adds to
    assert got is added and torch.equal(got, want)


def test_indices_outside_the_row():
    x, idx, _ = _inputs(10, 32, 4, torch.float32)
    idx[0, 0], idx[3, 1], idx[9, 3] = -1, 32, 1 << 30
    sdm.device_status()
    for k in (torch.int32, torch.int64):
        loss, counts = routing.balance(x.cuda(), idx.cuda().to(k))
        assert sdm.device_status() == sdm.SDM_DEV_BAD_INDEX
        assert torch.equal(counts.cpu().long(), ref.count(idx, 32)) and int(counts.sum()) == 37


def test_empty_calls():
    empty = torch.empty((0, 16), device="cuda")
    none = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    loss, counts, grad = routing.balance(empty, none, gradient=True)
    assert loss.tolist() == [0.0] and not counts.any() and counts.shape == (1, 16) and grad.shape == (0, 16)
    offsets = torch.zeros(4, dtype=torch.int32, device="cuda")
    loss, counts = routing.balance(empty, none, offsets=offsets)
    assert loss.tolist() == [0.0] * 3 and not counts.any()
    x = torch.randn(5, 16, device="cuda")
    idx = torch.zeros((5, 2), dtype=torch.int32, device="cuda")
    loss, counts, grad = routing.balance(x, idx, offsets=offsets, gradient=True)  # every token behind the last sequence
    assert loss.tolist() == [0.0] * 3 and not counts.any() and not grad.any()
    loss, counts, grad = routing.balance(x, idx, offsets=offsets[:1], gradient=True)
    assert loss.numel() == 0 and counts.shape == (0, 16) and not grad.any()


def test_same_bits_each_time_and_in_a_graph():
    x, idx, gen = _inputs(3000, 200, 6, torch.bfloat16)
    x, idx = x.cuda(), idx.cuda()
    offsets = torch.tensor([0, 100, 2900, 3000], dtype=torch.int32, device="cuda")
    want = [t.clone() for t in routing.balance(x, idx, offsets=offsets, gradient=True)]
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(routing.balance(x, idx, offsets=offsets, gradient=True), want))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        routing.balance(x, idx, offsets=offsets, gradient=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = routing.balance(x, idx, offsets=offsets, gradient=True)
    other, oidx, _ = _inputs(3000, 200, 6, torch.bfloat16, seed=9)
    for values, index in ((x.clone(), idx.clone()), (other.cuda(), oidx.cuda())):
        x.copy_(values)
        idx.copy_(index)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, routing.balance(x, idx, offsets=offsets, gradient=True)))


@pytest.mark.parametrize("n,tokens", ((16384, 140000), (256, 9000000)))
def test_more_than_32_bits_of_logits(n, tokens):
    """More than 2^31 logits, all alike: every row has the gradient (c - C / n) / (T C), the last as the first."""
    x = torch.zeros((tokens, n), dtype=torch.bfloat16, device="cuda")
    idx = torch.randint(0, n, (tokens, 2), device="cuda", dtype=torch.int32)
    loss, counts, grad = routing.balance(x, idx, gradient=True)
    assert torch.equal(counts[0].long(), torch.bincount(idx.view(-1).long(), minlength=n))
    total = 2 * tokens
    assert abs(float(loss) - 1) <= 200 * ref.STEP
    want = (counts[0].double().cpu() - total / n) / (tokens * float(total))
    moved = ref.STEP * ((counts[0].double().cpu() - total / n).abs() + total / n * ref.STEP) / (tokens * float(total)) * 2
    for t in (0, tokens // 2, (1 << 31) // n - 1, (1 << 31) // n, tokens - 1):
        ref.close(grad[t], want, moved + moved.mean(), f"row {t}", PARTS)
