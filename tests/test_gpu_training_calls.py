"""The training operators' calls: refusals of tensors on the GPU, given streams, the device status, threads at once."""

from __future__ import annotations

import threading

import pytest
import torch

from decode_state_gb300 import embedding, quant, routing, sdm

pytestmark = pytest.mark.gpu


def _sets():
    gen = torch.Generator(device="cuda").manual_seed(0)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    x = randn(3000, 96)
    chosen = torch.randint(0, 96, (3000, 4), generator=gen, device="cuda")
    tokens = torch.randint(0, 500, (20000,), generator=gen, device="cuda")
    return x, chosen, randn(500, 64), tokens, randn(20000, 64), randn(20000, 2)


def _calls():
    x, chosen, table, tokens, dout, w = _sets()
    idx = tokens[:, None].repeat(1, 2)
    return [
        ("balance", lambda s: list(routing.balance(x, chosen, gradient=True, stream=s))),
        ("lookup", lambda s: [embedding.lookup(table, tokens, stream=s)]),
        ("backward, few", lambda s: [embedding.backward(dout[:100], tokens[:100], 500, stream=s)]),
        ("backward, some", lambda s: [embedding.backward(dout[:5000], tokens[:5000], 500, stream=s)]),
        ("backward, many", lambda s: [embedding.backward(dout, tokens, 500, stream=s)]),
        ("rows", lambda s: [quant.gather_drows([(idx, w, dout)], 500, stream=s)]),
    ]


@pytest.mark.parametrize("at", range(6))
@pytest.mark.parametrize("as_handle", (False, True))
def test_memory_of_a_given_stream(at, as_handle):
    """Outputs and workspaces that a call makes for a stream are not memory that the current stream still writes."""
    name, call = _calls()[at]
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda.empty_cache()
    a = torch.ones((4096, 4096), device="cuda")
    held = [torch.empty(n, device="cuda") for n in [t.numel() for t in want] + [1 << 18, 1 << 20, 1 << 21]]
    torch.cuda.synchronize()
    for _ in range(40):
        a = (a @ a).mul_(1e-4)
    for t in held:
        t.fill_(12345.0)
    del held, t
    got = call(side.cuda_stream if as_handle else side)  # its inputs have been complete for long
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)), name


@pytest.mark.parametrize("at", range(6))
@pytest.mark.parametrize("handle", (0, 1, 2))
def test_handles_that_are_names(at, handle):
    name, call = _calls()[at]
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    for _ in range(3):
        got = call(handle)
        filler = [torch.full((1 << 21,), 7.0, device="cuda") for _ in range(2)]  # where the workspace may have been
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), name
        del filler


def test_threads_at_once():
    calls = _calls()
    want = [[t.clone() for t in call(None)] for _, call in calls]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        stream = torch.cuda.Stream()
        for r in range(10):
            name, call = calls[(i + r) % 6]
            got = call(stream)
            stream.synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, want[(i + r) % 6])):
                wrong.append(name)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(6)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_two_graphs_of_one_pool():
    """Graphs captured into one pool and replayed one after the other, many times, in either order."""
    calls = [c for _, c in _calls()]
    want = [[t.clone() for t in c(None)] for c in calls]
    torch.cuda.synchronize()
    graphs, got, pool = [], [], None
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            got.append(c(None))
        pool = g.pool()
        graphs.append(g)
    for order in ((0, 1, 2, 3, 4, 5), (5, 3, 1, 4, 2, 0)):
        for i in order:
            for t in got[i]:
                t.fill_(0)
            graphs[i].replay()
            assert all(torch.equal(a, b) for a, b in zip(got[i], want[i]))


def test_every_operator_raises_the_device_status():
    x, chosen, table, tokens, dout, w = _sets()
    bad, most = tokens.clone(), chosen.clone()
    bad[50], most[2, 1] = 500, 96
    sdm.device_status()
    for call in (lambda: routing.balance(x, most), lambda: embedding.lookup(table, bad), lambda: embedding.backward(dout, bad, 500),
                 lambda: embedding.backward(dout[:100], bad[:100], 500), lambda: embedding.backward(dout[:6000], bad[:6000], 500),
                 lambda: quant.gather_drows([(bad[:, None], w[:, :1].contiguous(), dout)], 500)):
        call()
        assert sdm.device_status() == sdm.SDM_DEV_BAD_INDEX
        assert sdm.device_status() == 0


def test_refusals():
    x, chosen, table, tokens, dout, w = _sets()
    offsets = torch.tensor([0, 3000], dtype=torch.int32, device="cuda")
    shape = [
        lambda: routing.balance(x, chosen[:10]), lambda: routing.balance(x, chosen.t()), lambda: routing.balance(x[:, ::2], chosen),
        lambda: routing.balance(x, chosen, w=w), lambda: routing.balance(x, chosen, base=tokens), lambda: routing.balance(x, chosen.cpu()),
        lambda: routing.balance(x, chosen, offsets=offsets[None]), lambda: routing.balance(x, chosen, offsets=offsets[:0]),
        lambda: routing.balance(x, chosen, add=x), lambda: routing.balance(x, chosen, out=x), lambda: routing.balance(x, chosen, dloss=x[0, :1]),
        lambda: routing.balance(x, chosen, gradient=True, add=x[:, :50]), lambda: routing.balance(x, chosen, gradient=True, out=x[:5]),
        lambda: routing.balance(x, chosen, gradient=True, dloss=x[0, :2]), lambda: routing.balance(x, chosen, loss=x[0, :3]),
        lambda: embedding.lookup(table, tokens.cpu()), lambda: embedding.lookup(table[:, ::2], tokens), lambda: embedding.lookup(table, tokens[::2]),
        lambda: embedding.lookup(table, tokens, out=dout[:5]), lambda: embedding.lookup(table, tokens, out=dout.cpu()),
        lambda: embedding.backward(dout, tokens[:5], 500), lambda: embedding.backward(dout, tokens, 500, accumulate=True),
        lambda: embedding.backward(dout, tokens, 500, out=table[:400]),
        lambda: embedding.backward(dout[:, ::2], tokens, 500), lambda: embedding.backward(dout.view(-1), tokens, 500),
        lambda: quant.gather_drows([(tokens, w, dout)], 500), lambda: quant.gather_drows([(chosen, w, dout)], 500),
        lambda: quant.gather_drows([(tokens[:, None], w[:, :1], dout)], 500), lambda: quant.gather_drows([(tokens.view(-1, 2), w[:10000], dout)], 500),
    ]
    for i, call in enumerate(shape):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"shape {i} was taken")
    kinds = [
        lambda: routing.balance(x.half(), chosen), lambda: routing.balance(x, chosen.float()), lambda: routing.balance(x, chosen, offsets=offsets.long()),
        lambda: routing.balance(x, chosen, w=torch.ones(chosen.shape, device="cuda", dtype=torch.bfloat16)), lambda: routing.balance(x, chosen, base=tokens[:3000].int()),
        lambda: routing.balance(x, chosen, counts=torch.zeros((1, 96), device="cuda")), lambda: routing.balance(x, chosen, gradient=True, add=x.bfloat16()),
        lambda: embedding.lookup(table.half(), tokens), lambda: embedding.lookup(table, tokens, dtype=torch.float16), lambda: embedding.lookup(table, tokens, dtype="bf16"),
        lambda: embedding.backward(dout, tokens.float(), 500), lambda: embedding.backward(dout, tokens, 500, dtype=torch.float64),
        lambda: quant.gather_drows([(tokens[:, None], w[:, :1].half(), dout)], 500), lambda: quant.gather_drows([(tokens[:, None], w[:, :1].contiguous(), dout.bfloat16())], 500),
    ]
    for i, call in enumerate(kinds):
        with pytest.raises(TypeError):
            call()
            pytest.fail(f"type {i} was taken")
    codes = [
        (lambda: routing.balance(x, chosen, gradient=True, out=x), -10), (lambda: routing.balance(x, chosen, counts=chosen.view(torch.int32).view(-1)[:96].view(1, 96)), -10),
        (lambda: embedding.lookup(table, tokens[:500], out=table), -10), (lambda: embedding.backward(table, tokens[:500], 500, out=table), -10),
        (lambda: embedding.backward(dout, tokens, 0), -7), (lambda: embedding.backward(dout, tokens, -1), -7),
        (lambda: embedding.backward(dout, tokens, 1 << 40), -7), (lambda: quant.gather_drows([(tokens[:, None], w[:, :1].contiguous(), dout)], 1 << 31), -7),
    ]
    for i, (call, code) in enumerate(codes):
        with pytest.raises(sdm.SDMError) as e:
            call()
        assert e.value.status == code, i
