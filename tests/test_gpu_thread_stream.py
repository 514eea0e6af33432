"""Calls for the stream of the thread (handle 2) beside a current stream of PyTorch's, which do not wait for each other: neither
the outputs nor the workspaces of a call are memory that the current stream still writes, or is given again too early."""

from __future__ import annotations

import threading

import pytest
import torch

from decode_state_gb300 import embedding, quant, routing

pytestmark = pytest.mark.gpu

THREAD = 2


def _calls():
    gen = torch.Generator(device="cuda").manual_seed(0)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    x, table, dout, w = randn(3000, 96), randn(500, 64), randn(40000, 64), randn(40000, 2)
    chosen = torch.randint(0, 96, (3000, 4), generator=gen, device="cuda")
    tokens = torch.randint(0, 500, (40000,), generator=gen, device="cuda")
    idx = tokens[:, None].repeat(1, 2)
    bank = quant.QuantBank.from_rows(randn(512, 128))
    slots = torch.randint(0, 512, (512, 8), generator=gen, device="cuda")
    return [
        ("balance", lambda s: list(routing.balance(x, chosen, gradient=True, stream=s))),
        ("lookup", lambda s: [embedding.lookup(table, tokens, stream=s)]),
        ("backward, few", lambda s: [embedding.backward(dout[:100], tokens[:100], 500, stream=s)]),
        ("backward, some", lambda s: [embedding.backward(dout[:5000], tokens[:5000], 500, stream=s)]),
        ("backward, many", lambda s: [embedding.backward(dout, tokens, 500, stream=s)]),
        ("rows", lambda s: [quant.gather_drows([(idx, w, dout)], 500, stream=s)]),
        ("route", lambda s: list(routing.route(x, 8, stream=s))),
        ("gather", lambda s: quant.gather(bank, [(slots, w[:2048].reshape(512, 8))], stream=s)),
        ("dequantize_rows", lambda s: [quant.dequantize_rows(bank, dtype=torch.float32, stream=s)]),
    ]


def _busy(a):
    for _ in range(40):
        a = (a @ a).mul_(1e-4)


@pytest.mark.parametrize("at", range(9))
def test_memory_that_the_current_stream_still_writes(at):
    name, call = _calls()[at]
    want = [t.clone() for t in call(None)]
    a = torch.ones((4096, 4096), device="cuda")
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        held = [torch.empty(n, device="cuda") for n in [t.numel() * t.element_size() // 4 for t in want] + [1 << 18, 1 << 20, 1 << 21]]
        torch.cuda.synchronize()
        _busy(a)
        for t in held:
            t.zero_()  # every word is a slot of the bank, if a call were to read it
        del held, t
        got = call(THREAD)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want)), name


@pytest.mark.parametrize("at", range(9))
def test_outputs_that_are_gone_before_the_call_is_done(at):
    name, call = _calls()[at]
    sizes = [t.numel() * t.element_size() // 4 for t in call(None)]
    a = torch.ones((4096, 4096), device="cuda")
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    with torch.cuda.stream(torch.cuda.ExternalStream(THREAD)):
        _busy(a)
    with torch.cuda.stream(side):
        call(THREAD)  # its outputs go at once
        filler = [torch.full((n,), 7.0, device="cuda") for n in sizes for _ in range(2)]
    torch.cuda.synchronize()
    assert all(bool((t == 7.0).all()) for t in filler), name


def test_outputs_given_need_no_wait():
    """A call that takes no memory runs beside the current stream."""
    table, tokens = torch.randn(500, 64, device="cuda"), torch.randint(0, 500, (2000,), device="cuda")
    out = torch.empty((2000, 64), device="cuda")
    a = torch.ones((4096, 4096), device="cuda")
    side, done = torch.cuda.Stream(), torch.cuda.Event()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        _busy(a)
        end = torch.cuda.Event()
        end.record()
        embedding.lookup(table, tokens, out=out, stream=THREAD)
    done.record(torch.cuda.ExternalStream(THREAD))
    done.synchronize()
    beside = not end.query()
    torch.cuda.synchronize()
    assert beside and torch.equal(out, table[tokens])


def test_captured_with_the_current_stream():
    """Both streams in one capture, forked and joined by the caller, and replayed."""
    table, tokens = torch.randn(500, 64, device="cuda"), torch.randint(0, 500, (20000,), device="cuda")
    dout = torch.randn(20000, 64, device="cuda")
    want = embedding.backward(dout, tokens, 500).clone()
    torch.cuda.synchronize()
    thread = torch.cuda.ExternalStream(THREAD)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        thread.wait_stream(torch.cuda.current_stream())
        got = embedding.backward(dout, tokens, 500, stream=THREAD)
        torch.cuda.current_stream().wait_stream(thread)
    for _ in range(2):
        got.fill_(0)
        graph.replay()
        assert torch.equal(got, want)


def test_banks_of_two_threads():
    """Two threads' streams go by the same handle: a bank that is gone in one is not the other's before its stream is done."""
    gen = torch.Generator(device="cuda").manual_seed(0)
    first, second = (torch.randn(4096, 128, generator=gen, device="cuda") for _ in range(2))
    want = quant.QuantBank.from_rows(second)
    a = torch.ones((4096, 4096), device="cuda")
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    made, finish = threading.Event(), threading.Event()

    def busy():
        with torch.cuda.stream(torch.cuda.ExternalStream(THREAD)):
            _busy(a)
        quant.QuantBank.from_rows(first, stream=THREAD)  # goes at once
        made.set()
        finish.wait(60)

    thread = threading.Thread(target=busy)
    thread.start()
    try:
        assert made.wait(60)
        got = quant.QuantBank.from_rows(second, stream=THREAD)
        torch.cuda.synchronize()
    finally:
        finish.set()
        thread.join()
    assert torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales)
