"""Outputs that a call makes for a stream it is given: their memory is free for that stream, whatever the current
stream still does with tensors that are gone."""

from __future__ import annotations

import pytest
import torch

from decode_state_gb300 import quant, routing

pytestmark = pytest.mark.gpu


def _busy_then_free(numel):
    """Work on the current stream that ends with writes to a tensor of this many float32, which is freed."""
    a = torch.ones((4096, 4096), device="cuda")
    t = torch.empty(numel, device="cuda")
    torch.cuda.synchronize()
    for _ in range(40):
        a = (a @ a).mul_(1e-4)
    t.fill_(12345.0)


def _calls():
    gen = torch.Generator(device="cuda").manual_seed(0)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    bank = quant.QuantBank.from_rows(randn(512, 128))
    x, idx = randn(1024, 64), torch.randint(0, 512, (512, 8), generator=gen, device="cuda")
    w, dout = randn(512, 8), randn(512, 128)
    at = torch.stack([torch.randperm(64, generator=gen, device="cuda")[:4] for _ in range(1024)])
    dw = randn(1024, 4)
    k_idx = torch.arange(512, device="cuda").view(64, 8)
    decode = (k_idx, torch.zeros(64, 8, device="cuda"), randn(64, 128), torch.ones(64, device="cuda"),
              torch.zeros(64, 1, device="cuda"), k_idx, randn(64, 8))  # a decode that leaves the bank as it is
    return [
        ("dequantize_rows", lambda s: [quant.dequantize_rows(bank, dtype=torch.float32, stream=s)]),
        ("gather", lambda s: quant.gather(bank, [(idx, w)], stream=s)),
        ("gather_dw", lambda s: quant.gather_dw(bank, [(idx, dout)], stream=s)),
        ("decode_step", lambda s: [quant.decode_step(bank, *decode, out_dtype=torch.float32, stream=s)]),
        ("route", lambda s: list(routing.route(x, 8, stream=s))),
        ("route_backward", lambda s: [routing.route_backward(x, at, dw, stream=s)]),
        ("from_rows", lambda s: [(b := quant.QuantBank.from_rows(dout, stream=s)).codes, b.scales]),
    ]


@pytest.mark.parametrize("as_handle", (False, True))
@pytest.mark.parametrize("at", range(7))
def test_outputs_are_not_memory_in_use(at, as_handle):
    name, call = _calls()[at]
    want = call(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    sizes = [t.numel() * t.element_size() // 4 for t in want]
    want = [t.clone() for t in want]
    torch.cuda.empty_cache()
    for n in sizes:
        _busy_then_free(n)
    got = call(side.cuda_stream if as_handle else side)  # its inputs have been complete for long
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)), name


@pytest.mark.parametrize("at", range(7))
@pytest.mark.parametrize("handle", (0, 1, 2))
def test_handles_that_are_names(at, handle):
    """The default stream's and the thread's own, which are no streams of PyTorch's."""
    name, call = _calls()[at]
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    got = call(handle)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)), name
