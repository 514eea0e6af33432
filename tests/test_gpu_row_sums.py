"""The embedding lookup, the table's gradient and the bank rows' gradient against plain forms in 64 bits.

Tolerances. A sum of m terms is m fused multiply-adds, the joins of the pieces it is cut into among them, of one rounding
of 2^-24 each, relative to the sum of the magnitudes at most; scaling it is one more, and so is adding to what was there.
Then one rounding to the output's type."""

from __future__ import annotations

import pytest
import torch

import train_reference as ref
from decode_state_gb300 import embedding, quant, sdm

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _bound(size, terms):
    return ref.STEP * size * (terms[:, None] + 12)  # 8 warps' joins, the tail, the scale, the addition


def _check_rows(got, ops, rows, before=None, **kw):
    sums, size, terms = ref.row_sums(ops, rows, **kw)
    if before is not None:
        sums, size = sums + before.double(), size + before.double().abs()
        untouched = terms == 0
        assert torch.equal(got.cpu()[untouched], before[untouched])
    else:
        assert not got.cpu()[terms == 0].any()
    ref.close(got, sums, _bound(size, terms), "sums")


def _tokens(count, rows, gen, skewed=True):
    if not skewed:
        return torch.randint(0, rows, (count,), generator=gen)
    rank = torch.exp(torch.rand(count, generator=gen, dtype=torch.float64) * torch.log(torch.tensor(rows + 1.0))).long() - 1
    return torch.randperm(rows, generator=gen)[rank.clamp(0, rows - 1)]


# ---------------------------------------------------------------- lookup

@pytest.mark.parametrize("hd", (1, 3, 8, 64, 100, 136, 264, 1024, 2048, 5000, 65536))
@pytest.mark.parametrize("table", (BF16, F32))
@pytest.mark.parametrize("out", (BF16, F32))
def test_lookup(hd, table, out):
    gen = torch.Generator().manual_seed(hd)
    rows, count = 50, 7 if hd > 2048 else 301
    t = torch.randn(rows, hd, generator=gen).to(table)
    tokens = torch.randint(0, rows, (count,), generator=gen)
    scale = 1.7 ** 0.5
    want = (t.float()[tokens] * torch.tensor(scale)).to(out)  # one float32 product, one rounding
    for it in (torch.int32, torch.int64):
        got = embedding.lookup(t.cuda(), tokens.cuda().to(it), scale=scale, dtype=out)
        assert got.dtype == out and torch.equal(got.cpu(), want)
    want[tokens == int(tokens[0])] = 0
    got = embedding.lookup(t.cuda(), tokens.cuda(), scale=scale, dtype=out, padding=int(tokens[0]))
    assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("shape", ((), (0,), (1,), (4, 0), (3, 5), (2, 3, 4)))
def test_lookup_shapes(shape):
    t = torch.randn(9, 24, device="cuda")
    tokens = torch.randint(0, 9, shape, device="cuda")
    got = embedding.lookup(t, tokens)
    assert got.shape == (*shape, 24) and got.dtype == F32 and torch.equal(got, t[tokens])
    out = torch.full((*shape, 24), 7.0, device="cuda")
    assert embedding.lookup(t, tokens, out=out) is out and torch.equal(out, t[tokens])


def test_lookup_outside_the_table():
    t = torch.randn(9, 40, device="cuda")
    tokens = torch.tensor([0, -1, 8, 9, 1 << 40, -100], device="cuda")
    sdm.device_status()
    got = embedding.lookup(t, tokens)
    assert sdm.device_status() == sdm.SDM_DEV_BAD_INDEX
    least = torch.full((3,), -(1 << 63), device="cuda")  # the number that stands for no padding in the C call
    assert not embedding.lookup(t, least).any() and sdm.device_status() == sdm.SDM_DEV_BAD_INDEX
    assert not embedding.backward(t[:3], least, 9).any() and sdm.device_status() == sdm.SDM_DEV_BAD_INDEX
    assert torch.equal(got[[0, 2]], t[[0, 8]]) and not got[[1, 3, 4, 5]].any()
    got = embedding.lookup(t, tokens[:3], padding=-1)  # a padding token outside the table is no error
    assert sdm.device_status() == 0 and not got[1].any()


@pytest.mark.parametrize("shift", (1, 2, 4))
@pytest.mark.parametrize("dtype", (BF16, F32))
def test_misaligned(shift, dtype):
    gen = torch.Generator().manual_seed(shift)
    rows, hd, count = 33, 64, 700
    wide = torch.randn(rows * hd + shift, generator=gen).to(dtype).cuda()
    t = wide[shift:].view(rows, hd)
    tokens = torch.randint(0, rows, (count,), generator=gen).cuda()
    out = torch.empty(count * hd + shift, dtype=dtype, device="cuda")[shift:].view(count, hd)
    assert torch.equal(embedding.lookup(t, tokens, out=out), t[tokens])
    dout = torch.randn(count * hd + shift, generator=gen).to(dtype).cuda()[shift:].view(count, hd)
    grad = torch.empty(rows * hd + shift, dtype=dtype, device="cuda")[shift:].view(rows, hd)
    embedding.backward(dout, tokens, rows, out=grad)
    _check_rows(grad, [(tokens.cpu()[:, None], None, dout.cpu())], rows)


# ---------------------------------------------------------------- the table's gradient

COUNTS = (0, 1, 2, 33, 511, 512, 513, 600, 4097, 8192, 8193, 9000, 40000)  # both sides of each path


@pytest.mark.parametrize("count", COUNTS)
@pytest.mark.parametrize("dtype,out", ((BF16, F32), (F32, BF16), (F32, F32), (BF16, BF16)))
@pytest.mark.parametrize("accumulate", (False, True))
def test_embedding_gradient(count, dtype, out, accumulate):
    gen = torch.Generator().manual_seed(count)
    rows, hd = 997, 72
    tokens = _tokens(count, rows, gen)
    dout = torch.randn(count, hd, generator=gen).to(dtype)
    before = torch.randn(rows, hd, generator=gen).to(out) if accumulate else None
    grad = None if before is None else before.clone().cuda()
    padding = int(tokens[-1]) if count else 5
    got = embedding.backward(dout.cuda(), tokens.cuda(), rows, scale=0.3, padding=padding, dtype=out, out=grad, accumulate=accumulate)
    assert got.dtype == out and (grad is None or got is grad)
    scale = float(torch.tensor(0.3, dtype=F32))
    _check_rows(got, [(tokens[:, None], None, dout)], rows, before, scale=scale, padding=padding)


@pytest.mark.parametrize("hd", (1, 2, 31, 64, 66, 128, 132, 256, 264, 700, 1024, 4100, 65536))
@pytest.mark.parametrize("dtype", (BF16, F32))
def test_embedding_widths(hd, dtype):
    gen = torch.Generator().manual_seed(hd)
    for count in (100, 700, 9000):
        if hd * count > 1 << 25:
            continue
        rows = 61
        tokens = _tokens(count, rows, gen)
        dout = torch.randn(count, hd, generator=gen).to(dtype)
        got = embedding.backward(dout.cuda(), tokens.cuda().to(torch.int32), rows)
        _check_rows(got, [(tokens[:, None], None, dout)], rows)


@pytest.mark.parametrize("rows", (1, 2, 255, 256, 257, 2047, 2048, 4095, 4096, 65535, 65536, 1 << 22, (1 << 22) + 1))
@pytest.mark.parametrize("count", (300, 3000, 20000))
def test_key_bits(rows, count):
    """Slots of every number of bits, on both sides of a power of two."""
    gen = torch.Generator().manual_seed(rows)
    tokens = torch.randint(0, rows, (count,), generator=gen)
    tokens[::7] = rows - 1
    dout = torch.randn(count, 4, generator=gen)
    got = embedding.backward(dout.cuda(), tokens.cuda(), rows)
    _check_rows(got, [(tokens[:, None], None, dout)], rows)


@pytest.mark.parametrize("count", (512, 8192, 8200, 100000))
@pytest.mark.parametrize("pattern", ("one", "two", "edges", "in order", "backwards", "all padding", "all but one padding"))
def test_runs(count, pattern):
    """Runs over many pieces, runs that end where a piece does, every entry a run; nothing to sum."""
    rows, hd, pad = 128 * 1024, 40, 77
    at = torch.arange(count)
    tokens = {"one": torch.full((count,), 5), "two": (at > count // 3).long() * 4000, "edges": at // 16, "in order": at, "backwards": count - 1 - at,
              "all padding": torch.full((count,), pad), "all but one padding": torch.full((count,), pad)}[pattern]
    if pattern == "all but one padding":
        tokens[count // 2] = 3
    dout = torch.randn(count, hd, generator=torch.Generator().manual_seed(1))
    got = embedding.backward(dout.cuda(), tokens.cuda(), rows, padding=pad)
    _check_rows(got, [(tokens[:, None], None, dout)], rows, padding=pad)


def test_tokens_outside_the_table():
    dout = torch.randn(700, 16, device="cuda")
    tokens = torch.randint(0, 9, (700,), device="cuda")
    tokens[::5], tokens[1::5] = -1, 9
    dout[::5], dout[1::5] = torch.nan, torch.inf
    for count in (20, 700):
        sdm.device_status()
        got = embedding.backward(dout[:count], tokens[:count], 9)
        assert sdm.device_status() == sdm.SDM_DEV_BAD_INDEX
        _check_rows(got, [(tokens[:count].cpu()[:, None], None, dout[:count].cpu().nan_to_num(0, 0, 0))], 9)


# ---------------------------------------------------------------- the bank rows' gradient

@pytest.mark.parametrize("tokens", (0, 1, 4, 12, 60, 400, 3000))
@pytest.mark.parametrize("widths", ((1,), (5,), (64, 32), (3, 256)))
@pytest.mark.parametrize("wdtype,out", ((BF16, F32), (F32, BF16)))
def test_gather_rows(tokens, widths, wdtype, out):
    gen = torch.Generator().manual_seed(tokens)
    rows, hd = 501, 36
    for chunk, valid, ragged in ((1, None, False), (4, 3, False), (4, None, True), (1, 0, False)):
        if tokens % chunk:
            continue
        cv = torch.randint(0, chunk + 1, (tokens // chunk,), generator=gen).to(torch.int32) if ragged else None
        ops = []
        for w in widths:
            weight = torch.randn(tokens, w, generator=gen).to(wdtype)
            weight[torch.rand(tokens, w, generator=gen) < 0.1] = 0
            ops.append((_tokens(tokens * w, rows, gen).view(tokens, w), weight, torch.randn(tokens, hd, generator=gen)))
        got = quant.gather_drows([tuple(t.cuda() for t in o) for o in ops], rows, chunk=chunk, valid=valid,
                                 chunk_valid=None if cv is None else cv.cuda(), dtype=out)
        _check_rows(got, ops, rows, chunk=chunk, valid=valid, chunk_valid=cv)


@pytest.mark.parametrize("tokens", (40, 2000))
def test_left_out_whatever_they_hold(tokens):
    """Padding, weights of 0 and indices outside the bank beside dout and weights that are no numbers."""
    gen = torch.Generator().manual_seed(tokens)
    rows, hd, width, chunk = 100, 24, 6, 8
    idx, w = torch.randint(0, rows, (tokens, width), generator=gen), torch.randn(tokens, width, generator=gen)
    dout = torch.randn(tokens, hd, generator=gen)
    pad = torch.arange(tokens) % chunk >= 5
    dout[pad], w[pad] = torch.nan, torch.inf
    dout[2], w[2] = torch.inf, 0.0
    dout[1], idx[1] = torch.nan, -3
    w[3, 2], idx[3, 2] = torch.nan, rows
    sdm.device_status()
    got = quant.gather_drows([(idx.cuda(), w.cuda(), dout.cuda())], rows, chunk=chunk, valid=5)
    assert sdm.device_status() == sdm.SDM_DEV_BAD_INDEX
    clean = dout.nan_to_num(0, 0, 0)
    _check_rows(got, [(idx, w.nan_to_num(0, 0, 0), clean)], rows, chunk=chunk, valid=5)


def test_agrees_with_the_gather():
    """<drows, bank> = <dout, gather>: both are the sum over all entries of w * <dout, row>."""
    gen = torch.Generator().manual_seed(3)
    rows, hd, tokens = 3000, 128, 512
    bank = torch.randn(rows, hd, generator=gen).cuda()
    ops = [(torch.randint(0, rows, (tokens, w), generator=gen).cuda(), torch.randn(tokens, w, generator=gen).cuda()) for w in (16, 5)]
    douts = [torch.randn(tokens, hd, generator=gen).cuda() for _ in ops]
    outs, _ = sdm.gather(bank, ops, chunk=1, with_stash=False)
    drows = quant.gather_drows([(i, w, d) for (i, w), d in zip(ops, douts)], rows)
    a = (drows.double() * bank.double()).sum()
    b = sum((o.double() * d.double()).sum() for o, d in zip(outs, douts))
    size = sum((d.double().abs()[:, None] * w.double().abs()[..., None] * bank.double()[i].abs()).sum() for (i, w), d in zip(ops, douts))
    assert abs(float(a - b)) <= 64 * ref.STEP * float(size)


def test_sums_far_into_a_large_gradient():
    """A gradient of more than 2^31 elements: rows on both sides of where 32 bits of an offset end."""
    rows, hd = (1 << 24) + 5, 256
    at = torch.tensor([0, (1 << 23) - 1, 1 << 23, (1 << 24) - 1, 1 << 24, rows - 1])
    tokens = at.repeat(200)
    gen = torch.Generator().manual_seed(0)
    dout = torch.randn(len(tokens), hd, generator=gen)
    grad = torch.full((rows, hd), 3.0, dtype=BF16, device="cuda")
    embedding.backward(dout.cuda(), tokens.cuda(), rows, out=grad)
    sums, size, terms = ref.row_sums([(torch.arange(6).repeat(200)[:, None], None, dout)], 6)
    ref.close(grad[at.cuda()], sums, _bound(size, terms), "sums")
    assert int((grad != 0).any(1).sum()) == 6
    table = torch.zeros((rows, hd), dtype=BF16, device="cuda")
    table[at.cuda()] = torch.arange(1, 7, device="cuda", dtype=BF16)[:, None]
    assert torch.equal(embedding.lookup(table, at.cuda())[:, 0].float().cpu(), torch.arange(1, 7).float())


@pytest.mark.parametrize("count", (300, 5000, 30000))
def test_same_bits_each_time_and_in_a_graph(count):
    gen = torch.Generator().manual_seed(count)
    tokens, dout = _tokens(count, 500, gen).cuda(), torch.randn(count, 96, generator=gen).cuda()
    want = embedding.backward(dout, tokens, 500).clone()
    for _ in range(5):
        assert torch.equal(embedding.backward(dout, tokens, 500), want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = embedding.backward(dout, tokens, 500)
    graph.replay()
    assert torch.equal(got, want)
    dout.mul_(2)
    tokens.copy_(_tokens(count, 500, gen))
    graph.replay()
    assert torch.equal(got, embedding.backward(dout, tokens, 500))


def test_two_streams_at_once():
    """Calls on two streams have workspaces of their own."""
    gen = torch.Generator().manual_seed(5)
    sets = [(torch.randn(30000, 64, generator=gen).cuda(), _tokens(30000, 700, gen).cuda()) for _ in range(2)]
    want = [embedding.backward(d, t, 700).clone() for d, t in sets]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):
        got = [embedding.backward(d, t, 700, stream=s) for (d, t), s in zip(sets, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_lookup_of_more_than_32_bits():
    """An output of more than 2^32 elements."""
    hd, count = 2048, 2200000
    table = torch.randn(50, hd, device="cuda").bfloat16()
    tokens = torch.randint(0, 50, (count,), device="cuda", dtype=torch.int32)
    out = embedding.lookup(table, tokens)
    for at in (0, (1 << 31) // hd - 1, (1 << 31) // hd, (1 << 32) // hd - 1, (1 << 32) // hd, count - 1):
        assert torch.equal(out[at], table[tokens[at]])
    dout = out[-3000000000 // hd:]  # the gradient of the last rows, from an address far into a tensor
    got = embedding.backward(dout, tokens[-len(dout):], 50)
    times = torch.bincount(tokens[-len(dout):].long(), minlength=50).double()
    want = times[:, None] * table.double()  # each of the sums is of equal terms, bf16 by whole numbers
    assert float((got.double() - want).abs().max()) <= float((times[:, None] * ref.STEP * want.abs()).max())
