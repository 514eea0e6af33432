"""The training operators where their kernels change: on both sides of every change of path, with several rows and
sequences for each team, and in the passes of the sort that few entries and few slots do not reach.

Tolerances as in test_gpu_balance and test_gpu_row_sums."""

from __future__ import annotations

import pytest
import torch

import train_reference as ref
from decode_state_gb300 import embedding, quant, routing, sdm

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
PARTS = 200.0


# ---------------------------------------------------------------- balance

def _cuts(tokens, sequences, gen, inside=False):
    """Offsets of so many sequences, some empty; `inside`: with tokens before the first and behind the last."""
    cuts = torch.randint(0, tokens + 1, (sequences + 1,), generator=gen).sort().values
    if not inside:
        cuts[0], cuts[-1] = 0, tokens
    return cuts.to(torch.int32)


def _balance(tokens, n, k, dtype, score, sequences, *, inside=False, add=False, pad=0, seed=0):
    gen = torch.Generator().manual_seed(seed)
    x = (torch.randn(tokens, n, generator=gen) * 2 + torch.randn(n, generator=gen) * 0.5).to(dtype)
    idx = torch.randint(0, n, (tokens, k), generator=gen)
    offsets = None if sequences is None else _cuts(tokens, sequences, gen, inside)
    dloss = torch.randn(1 if sequences is None else sequences, generator=gen)
    more = (torch.randn(tokens, n, generator=gen) * 1e-3).to(dtype) if add else None
    rows = torch.zeros((tokens, n + pad), dtype=dtype, device="cuda")[:, :n]
    rows.copy_(x)
    args = dict(score=score, offsets=None if offsets is None else offsets.cuda(), scale=0.8)
    sdm.device_status()
    loss, counts, grad = routing.balance(rows, idx.cuda(), gradient=True, dloss=dloss.cuda(), add=None if more is None else more.cuda(), **args)
    alone, same = routing.balance(rows, idx.cuda(), **args)
    assert sdm.device_status() == 0
    want = ref.count(idx, n, offsets=offsets)
    assert torch.equal(counts.cpu().long(), want) and torch.equal(same, counts)
    l64, g64, moved_l, moved_g = ref.balance(x, want, score=score, offsets=offsets, scale=0.8, dloss=dloss, add=more)
    ref.close(loss, l64, moved_l, "loss", PARTS)
    ref.close(alone, l64, moved_l, "loss without gradient", PARTS)
    if add:
        moved_g = moved_g + ref.STEP * g64.abs() / PARTS  # one more sum
    ref.close(grad, g64, moved_g, "gradient", PARTS)


@pytest.mark.parametrize("n,tokens,sequences", ((24, 200_001, 5000), (24, 200_001, 3), (100, 60_000, 40), (256, 70_001, 3000), (256, 30_000, 5),
                                                (500, 20_000, 700)))
@pytest.mark.parametrize("dtype,score", ((BF16, "sigmoid"), (F32, "softmax")))
def test_several_rows_and_sequences_a_team(n, tokens, sequences, dtype, score):
    _balance(tokens, n, 3, dtype, score, sequences, inside=sequences % 2 == 1, add=sequences > 100, seed=n + sequences)


@pytest.mark.parametrize("n,tokens,sequences", ((700, 9000, 400), (1024, 6001, 3), (2000, 5000, 1500), (2050, 5000, 60), (5000, 2500, 7),
                                                (8192, 2000, 300), (9000, 1500, 20), (30_000, 700, 9), (50_000, 1000, 5)))
@pytest.mark.parametrize("dtype,score", ((BF16, "softmax"), (F32, "sigmoid")))
@pytest.mark.parametrize("pad", (0, 1))
def test_several_rows_and_sequences_a_block(n, tokens, sequences, dtype, score, pad):
    """`pad` 1: rows that start anywhere."""
    _balance(tokens, n, 4, dtype, score, sequences, inside=sequences < 100, add=pad == 1, pad=pad, seed=n + pad)


@pytest.mark.parametrize("tokens,n,k,sequences", ((4096, 16, 2, 4096), (4096, 16, 2, 1000), (512, 128, 4, 512), (128, 512, 5, 40), (2048, 32, 4, 100),
                                                  (65536, 1, 1, 30), (2730, 24, 3, 4097), (4097, 16, 2, 20), (4096, 16, 2, 32), (2048, 32, 4, 32), (256, 256, 32, 33),
                                                  (1024, 16, 4, 1), (1024, 16, 1, 1), (1025, 16, 1, 1), (2048, 16, 4, 2), (1000, 64, 8, 31), (500, 128, 9, 1)))
@pytest.mark.parametrize("score", ("softmax", "sigmoid"))
def test_one_launch_and_four(tokens, n, k, sequences, score):
    """The largest calls of one launch, a cluster for each sequence, and calls beyond them."""
    _balance(tokens, n, k, F32, score, sequences, inside=sequences > 1, add=True, seed=sequences)


# ---------------------------------------------------------------- sums of rows

def _bound(size, terms):
    return ref.STEP * size * (terms[:, None] + 12)  # 8 warps' joins, the tail, the scale, the addition


def _check(got, ops, rows, before=None, **kw):
    sums, size, terms = ref.row_sums(ops, rows, **kw)
    if before is not None:
        assert torch.equal(got.cpu()[terms == 0], before[terms == 0])
        sums, size = sums + before.double(), size + before.double().abs()
    else:
        assert not got.cpu()[terms == 0].any()
    ref.close(got, sums, _bound(size, terms), "sums")


def _tokens(count, rows, gen):
    """Skewed: the first slots of some order come most often."""
    rank = (torch.rand(count, generator=gen, dtype=torch.float64) ** 4 * rows).long().clamp_(0, rows - 1)
    return torch.randperm(rows, generator=gen)[rank]


@pytest.mark.parametrize("count", (512, 513, 16384, 16385, 32768, 32769, 131072, 131073, 1 << 20, (1 << 20) + 1))
@pytest.mark.parametrize("rows", (997, 1 << 17))
@pytest.mark.parametrize("accumulate", (False, True))
def test_both_sides_of_each_path(count, rows, accumulate):
    gen = torch.Generator().manual_seed(count + rows)
    tokens, dout = _tokens(count, rows, gen), torch.randn(count, 12, generator=gen)
    before = torch.randn(rows, 12, generator=gen) if accumulate else None
    got = embedding.backward(dout.cuda(), tokens.cuda(), rows, padding=int(tokens[3]), out=None if before is None else before.clone().cuda(),
                             accumulate=accumulate)
    _check(got, [(tokens[:, None], None, dout)], rows, before, padding=int(tokens[3]))


@pytest.mark.parametrize("rows", (1 << 11, (1 << 11) + 1, 1 << 17, 1 << 20, 1 << 22, (1 << 22) + 1))
@pytest.mark.parametrize("count", (40_000, 200_000, 1_200_000))
@pytest.mark.parametrize("dtype,out", ((BF16, F32), (F32, BF16)))
def test_passes_of_the_sort(rows, count, dtype, out):
    """One, two and three passes by launches, in tiles of both sizes."""
    gen = torch.Generator().manual_seed(rows + count)
    tokens, dout = torch.randint(0, rows, (count,), generator=gen), torch.randn(count, 3, generator=gen).to(dtype)
    tokens[::9] = rows - 1
    got = embedding.backward(dout.cuda(), tokens.cuda(), rows, dtype=out)
    _check(got, [(tokens[:, None], None, dout)], rows)


@pytest.mark.parametrize("rows", (3000, 1 << 20, (1 << 22) + 5))
@pytest.mark.parametrize("accumulate", (False, True))
def test_many_entries_of_a_gather(rows, accumulate):
    """Two operands, padding, weights of zero, in tiles of 4096 entries."""
    gen = torch.Generator().manual_seed(rows)
    chunks, chunk, hd = 4500, 16, 3
    tokens = chunks * chunk
    valid = torch.randint(0, chunk + 1, (chunks,), generator=gen).to(torch.int32)
    ops = []
    for width in (21, 4):
        w = torch.randn(tokens, width, generator=gen)
        w[torch.rand(tokens, width, generator=gen) < 0.2] = 0
        ops.append((_tokens(tokens * width, rows, gen).view(tokens, width), w, torch.randn(tokens, hd, generator=gen)))
    before = torch.randn(rows, hd, generator=gen) if accumulate else None
    got = quant.gather_drows([tuple(t.cuda() for t in o) for o in ops], rows, chunk=chunk, chunk_valid=valid.cuda(),
                             out=None if before is None else before.clone().cuda(), accumulate=accumulate)
    _check(got, ops, rows, before, chunk=chunk, chunk_valid=valid)


@pytest.mark.parametrize("rows", (300, 1 << 20))
def test_more_tiles_than_a_scan_keeps(rows):
    """More than 2048 tiles: the running sums of a digit are read again."""
    count = 2048 * 4096 + 4097
    gen = torch.Generator().manual_seed(rows)
    tokens, dout = torch.randint(0, rows, (count,), generator=gen), torch.randint(-4, 5, (count, 2), generator=gen).to(BF16)
    got = embedding.backward(dout.cuda(), tokens.cuda(), rows)
    want = torch.zeros((rows, 2), dtype=torch.float64).index_add_(0, tokens, dout.double())
    assert torch.equal(got.cpu().double(), want)  # whole numbers far below 2^24


def test_most_entries():
    """2^31 - 1 entries. Token t is of row t mod 2^22, every 1024th of row 5, and brings one where bit 22 of t is set."""
    rows, count = 1 << 22, (1 << 31) - 1
    tokens = torch.empty(count + 1, dtype=torch.int32, device="cuda")
    dout = torch.empty((count + 1, 1), dtype=BF16, device="cuda")
    each = torch.arange(rows, dtype=torch.int32, device="cuda")
    each[::1024] = 5
    for m in range(512):
        tokens[m << 22:(m + 1) << 22] = each
        dout[m << 22:(m + 1) << 22] = m & 1
    sdm.device_status()
    got = embedding.backward(dout[:count], tokens[:count], rows)
    assert sdm.device_status() == 0
    want = torch.full((rows,), 256.0, device="cuda")
    want[::1024] = 0
    want[5] += 1 << 20
    want[-1] -= 1  # the token that is left out
    assert torch.equal(got[:, 0], want)


@pytest.mark.parametrize("count,rows", ((40_000, 700), (300_000, 1 << 18), (1_100_000, 1 << 12)))
def test_launches_of_the_sort_in_graphs_and_on_two_streams(count, rows):
    gen = torch.Generator().manual_seed(count)
    sets = [(torch.randn(count, 24, generator=gen).cuda(), _tokens(count, rows, gen).cuda()) for _ in range(2)]
    want = [embedding.backward(d, t, rows).clone() for d, t in sets]
    for (d, t), first in zip(sets, want):
        assert torch.equal(embedding.backward(d, t, rows), first)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):
        got = [embedding.backward(d, t, rows, stream=s) for (d, t), s in zip(sets, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    dout, tokens = sets[0][0].clone(), sets[0][1].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = embedding.backward(dout, tokens, rows)
    for (d, t), first in zip(sets, want):
        dout.copy_(d)
        tokens.copy_(t)
        graph.replay()
        assert torch.equal(out, first)
