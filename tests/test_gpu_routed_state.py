"""The routed decode state: its calls against the operators one by one and against 64-bit formulas.

Tolerances, fixed before the first run: readings by ``read`` (reads + 4) eps of their terms; the logits'
gradient 128 eps of the magnitudes that make it up, those of dw being (hd + 6) eps of its terms.
"""

from __future__ import annotations

import importlib.util
import os

import numpy as np
import pytest
import quant_reference as ref
import torch
from quant_reference import EPS

from decode_state_gb300 import quant, routing, sdm
from decode_state_gb300.state import RoutedLayerState

pytestmark = pytest.mark.gpu


def _randn(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).cuda()


def _state(streams=5, slots=70, hd=72, format="int8", **router):
    bank = quant.QuantBank.from_rows(_randn(streams * slots, hd, seed=1), group=64, format=format)
    return RoutedLayerState(bank, streams, writes=9, reads=13, **router)


def _inputs(s, *lead, seed=2):
    return (_randn(*lead, s.streams, s.slots, seed=seed), _randn(*lead, s.streams, s.memory.hd, seed=seed + 1),
            torch.sigmoid(_randn(*lead, s.streams, seed=seed + 2)), -0.1 * _randn(*lead, s.streams, 1, seed=seed + 3).abs(),
            _randn(*lead, s.streams, s.slots, seed=seed + 4))


@pytest.mark.parametrize("format", ("int8", "fp8"))
def test_steps_are_the_steps_one_by_one(format):
    one, many = _state(format=format), _state(format=format, seq_len=3)
    x = _inputs(one, 6)
    got = many.steps(*x)
    want = torch.stack([one.step(*(a[t] for a in x)) for t in range(6)])
    assert torch.equal(got, want) and torch.equal(one.rows(), many.rows())
    assert (one.cache_len, many.cache_len) == (6, 9)


def test_step_is_route_and_decode():
    a, b = _state(score="sigmoid", scale=0.5), _state()
    k, v, beta, g, q = _inputs(a)
    got = a.step(k, v, beta, g, q, out_dtype=torch.float32)
    base = torch.arange(5, dtype=torch.int32, device="cuda") * 70
    ki, kw = routing.route(k, 9, score="sigmoid", scale=0.5, base=base)
    qi, qw = routing.route(q, 13, score="sigmoid", scale=0.5, base=base)
    want = quant.decode_step(b.memory, ki, kw, v, beta, g, qi, qw, out_dtype=torch.float32)
    assert torch.equal(got, want) and torch.equal(a.memory.codes, b.memory.codes)


@pytest.mark.parametrize("format", ("int8", "fp8", "int4"))
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True)])
def test_reading_and_its_gradient(format, score, renorm):
    s = _state(format=format, score=score, renorm=renorm)
    q = _randn(5, 70, seed=8)
    out, idx, w = s.read(q)
    rows = torch.from_numpy(ref.values(s.memory.codes.cpu().numpy(), s.memory.scales.cpu().numpy(), 72, 64, format))
    terms = w.cpu().double()[..., None] * rows[idx.cpu()]
    assert bool(((out.cpu().double() - terms.sum(1)).abs() <= 17 * EPS * terms.abs().sum(1)).all())
    local = (idx - 70 * torch.arange(5, device="cuda")[:, None]).cpu().numpy()
    want, _ = ref.route(q.cpu().numpy(), 13, score)
    assert np.array_equal(local, want)
    dout = _randn(5, 72, seed=9)
    got = s.read_backward(q, idx, dout).cpu().double().numpy()
    dterms = dout.cpu().double()[:, None] * rows[idx.cpu()]
    grad, size = ref.route_backward(q.cpu().numpy(), local, dterms.sum(2).numpy(), score, renorm, 1.0)
    _, loose = ref.route_backward(q.cpu().numpy(), local, dterms.abs().sum(2).numpy(), score, renorm, 1.0)
    assert (np.abs(got - grad) <= 128 * EPS * size + 78 * EPS * loose).all()


def test_load_reset_and_refusals():
    s = _state()
    rows = _randn(350, 72, seed=5)
    assert s.load_(rows, 11).cache_len == 11
    same = quant.QuantBank.from_rows(rows, group=64)
    assert torch.equal(s.rows(torch.float32), quant.dequantize_rows(same, dtype=torch.float32))
    s.reset()
    assert s.cache_len == 0 and not s.rows().any()
    with pytest.raises(ValueError, match="do not divide"):
        RoutedLayerState(s.memory, 4, writes=1, reads=1)
    with pytest.raises(ValueError, match="set by the state"):
        RoutedLayerState(s.memory, 5, writes=1, reads=1, base=None)
    with pytest.raises(ValueError, match="logits must be"):
        s.read(_randn(4, 70))


def test_example_runs_and_learns():
    path = os.path.join(os.path.dirname(__file__), "..", "examples", "routed_memory.py")
    spec = importlib.util.spec_from_file_location("routed_memory", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    result = module.main(streams=8, slots=64, hd=32, prompt=4, tokens=2, rounds=30)
    assert all(torch.isfinite(r.float()).all() for r in result["readings"])
    assert result["losses"][-1] < result["losses"][0]
    assert sdm.device_status() == 0
