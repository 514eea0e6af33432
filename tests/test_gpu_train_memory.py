"""The training operators together: a layer from tokens to readings and back, against automatic differentiation in 64
bits, and the routed state's gradients of rows and balance.

Tolerances. The layer's gradients are sums of products of quantities that are right to a few hundred roundings of 2^-24
each (matrix products of up to 1000 float32 terms among them), relative to the sums of the magnitudes: 2^-24 * 2000 of the
largest gradient's scale bounds them."""

from __future__ import annotations

import os
import sys

import pytest
import torch

import train_reference as ref
from decode_state_gb300 import quant, routing
from decode_state_gb300.state import RoutedLayerState

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import train_memory  # noqa: E402

pytestmark = pytest.mark.gpu


def _layer(table, router, bank, tokens, target, idx, counts, scale, balance, score, offsets):
    """The example's loss in float64, its choices and counts fixed."""
    x = table[tokens] * scale * (tokens != train_memory.PADDING)[:, None]
    logits = x @ router
    s = torch.softmax(logits, 1) if score == "softmax" else torch.sigmoid(logits)
    p = s / s.sum(1, keepdim=True)
    w = s.gather(1, idx)
    out = ((w / w.sum(1, keepdim=True))[..., None] * bank[idx]).sum(1)
    loss = ((out - target) ** 2).mean()
    for q, (a, b) in enumerate(ref.sequences(len(tokens), offsets)):
        if b > a:
            loss = loss + balance * router.shape[1] / ((b - a) * counts[q].sum()) * (p[a:b] @ counts[q].double()).sum()
    return loss


@pytest.mark.parametrize("score", ("softmax", "sigmoid"))
@pytest.mark.parametrize("tokens,slots,hd,reads", ((40, 30, 20, 4), (600, 100, 64, 8), (700, 700, 33, 16)))
def test_gradients_of_a_layer(score, tokens, slots, hd, reads):
    gen = torch.Generator().manual_seed(tokens)
    randn = lambda *shape: torch.randn(shape, generator=gen)  # noqa: E731
    table, router, bank, target = randn(90, 16) / 4, randn(16, slots) / 2, randn(slots, hd), randn(tokens, hd)
    batch = torch.randint(0, 90, (tokens,), generator=gen)
    offsets = torch.tensor([0, tokens // 3, tokens // 3, tokens - 5], dtype=torch.int32)
    got = train_memory.gradients(table.cuda(), router.cuda(), bank.cuda(), batch.cuda(), target.cuda(), reads=reads, scale=2.0, balance=0.5,
                                 score=score, offsets=offsets.cuda())
    idx = got["idx"].cpu().long()
    assert torch.equal(got["counts"].cpu().long(), ref.count(idx, slots, offsets=offsets))
    params = [t.double().requires_grad_() for t in (table, router, bank)]
    loss = _layer(*params, batch, target.double(), idx, got["counts"].cpu(), 2.0, 0.5, score, offsets)
    assert abs(float(loss.detach()) - float(got["loss"])) <= 2000 * ref.STEP * float(loss.detach())
    for name, grad in zip(("table", "router", "bank"), torch.autograd.grad(loss, params)):
        assert float((got[name].cpu().double() - grad).abs().max()) <= 2000 * ref.STEP * float(grad.abs().max()), name


def test_example_runs():
    result = train_memory.main(tokens=200, vocabulary=300, slots=64, hd=32, reads=4, rounds=3)
    assert len(result["losses"]) == 3 and all(torch.isfinite(torch.tensor(result["losses"])))
    assert result["counts"].shape == (2, 64) and int(result["counts"].sum()) == 800


def test_a_training_step_in_a_graph():
    """The whole pass captured, replayed on new tokens, while an eager one runs between."""
    gen = torch.Generator().manual_seed(0)
    randn = lambda *shape: torch.randn(shape, generator=gen).cuda()  # noqa: E731
    args = [randn(50, 16), randn(16, 40), randn(40, 24), torch.randint(0, 50, (1000,), generator=gen).cuda(), randn(1000, 24)]
    kw = dict(reads=4, offsets=torch.tensor([0, 300, 1000], dtype=torch.int32, device="cuda"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        train_memory.gradients(*args, **kw)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = train_memory.gradients(*args, **kw)
    for seed in (1, 2):
        args[3].copy_(torch.randint(0, 50, (1000,), generator=torch.Generator().manual_seed(seed)))
        want = train_memory.gradients(*args, **kw)
        graph.replay()
        for name in want:
            assert torch.equal(got[name], want[name]), name


@pytest.mark.parametrize("format", ("int8", "fp8"))
def test_routed_state(format):
    gen = torch.Generator().manual_seed(2)
    S, P, hd, k = 5, 48, 32, 6
    randn = lambda *shape: torch.randn(shape, generator=gen).cuda()  # noqa: E731
    state = RoutedLayerState(quant.QuantBank.from_rows(randn(S * P, hd), group=32, format=format), S, writes=4, reads=k, score="sigmoid")
    logits, dout = randn(S, P), randn(S, hd)
    out, idx, w = state.read(logits)
    got = state.rows_gradient(idx, w, dout)
    sums, size, terms = ref.row_sums([(idx.cpu(), w.cpu(), dout.cpu())], S * P)
    ref.close(got, sums, ref.STEP * size * (terms[:, None] + 12), "rows")
    more = state.rows_gradient(idx, w, dout, out=got.clone(), accumulate=True)
    assert torch.equal(more, 2 * got)
    # one token a stream, and three
    for lead in ((), (3,)):
        x = randn(*lead, S, P)
        chosen, weights = state.choose(x, k)
        add = randn(*lead, S, P) * 1e-3
        loss, counts, grad = state.balance(x, chosen, weights, scale=2.0, gradient=True, add=add)
        places = (chosen.cpu() - torch.arange(S)[:, None] * P).reshape(-1, k)
        want = ref.count(places, P)
        assert torch.equal(counts.cpu().long(), want) and grad.shape == x.shape
        l64, g64, moved_l, moved_g = ref.balance(x.cpu().reshape(-1, P), want, score="sigmoid", scale=2.0, add=add.cpu().reshape(-1, P))
        ref.close(loss, l64, moved_l, "loss", 200)
        ref.close(grad.reshape(-1, P), g64, moved_g + ref.STEP * g64.abs() / 200, "gradient", 200)
        alone = state.balance(x, chosen, weights, scale=2.0)
        assert len(alone) == 2 and torch.equal(alone[0], loss) and torch.equal(alone[1], counts)
    with pytest.raises(ValueError):
        state.balance(logits[:, :-1], idx)
    with pytest.raises(ValueError):
        state.balance(logits, idx[:3])


def test_route_then_balance_of_filled_entries():
    """Entries that only filled up where groups left too few are not counted, by the router's own weights."""
    x = torch.full((4, 16), -torch.inf, device="cuda")
    x[:, :3] = torch.randn(4, 3, device="cuda")
    idx, w = routing.route(x, 5)
    loss, counts = routing.balance(x, idx, w=w)
    assert int(counts.sum()) == 12 and counts[0, :3].tolist() == [4, 4, 4]
    assert int(routing.balance(x, idx)[1].sum()) == 20
