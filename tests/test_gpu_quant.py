"""Quantised banks on the GPU: written, read back, gathered (with the weights' gradient) and decoded,
against plain implementations.

Tolerances, fixed before the first run:
  codes, scales   bit-identical: their definition is a float32 division, product and rounding
  read back       bit-identical to the float32 product, rounded once
  gather          (N + 4) eps sum_n |w row|: N fma roundings, the product w * scale, a join of four sums
  gradient        (hd + 6) eps sum_c |dout row|, and one rounding to bfloat16 (2^-8 of the value)
  decode, rows    half a step of the format around the 64-bit value, plus the float32 error below
  decode, out     the gather's, over the rows that the kernel itself wrote
"""

from __future__ import annotations

import numpy as np
import pytest
import quant_reference as ref
import torch
from quant_reference import EPS

from decode_state_gb300 import quant, sdm

pytestmark = pytest.mark.gpu

FORMATS = ("int8", "fp8", "int4")
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _rows(n, hd, seed, dtype=torch.float32):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((n, hd), generator=gen) * torch.exp(2 * torch.randn((n, 1), generator=gen))
    return x.to(dtype)


def _bank(n, hd, group, fmt, seed=0):
    """(a QuantBank on the GPU, its float64 rows)."""
    codes, scales = ref.quantise(_rows(n, hd, seed).numpy(), group, fmt)
    bank = quant.QuantBank(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), hd, group=group, format=fmt)
    return bank, ref.values(codes, scales, hd, group, fmt)


def _same(a, b):
    return np.array_equal(a.cpu().numpy().view(np.uint8), np.ascontiguousarray(b).view(np.uint8))


@pytest.fixture(autouse=True)
def _clean_status():
    sdm.device_status()
    yield
    assert sdm.device_status() == 0


# ---------------------------------------------------------------- rows in and out

@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("n,hd,group", [(1, 1, 32), (3, 31, 32), (257, 64, 64), (65, 128, 128), (64, 136, 64),
                                        (33, 300, 128), (5, 1000, 32), (2, 4113, 128)])
def test_rows_are_stored_as_defined(fmt, dtype, n, hd, group):
    x = _rows(n, hd, hd, DTYPES[dtype])
    codes, scales = ref.quantise(x.float().numpy(), group, fmt)
    bank = quant.QuantBank.from_rows(x.cuda(), group=group, format=fmt)
    assert _same(bank.scales, scales)
    assert _same(bank.codes, codes)
    for out in ("bf16", "f32"):
        # the float32 product scale * code, rounded once; code and scale are exact in float32
        y32 = (ref.values(codes, np.ones_like(scales), hd, group, fmt).astype(np.float32)
               * scales[:, np.arange(hd) // group])
        got = quant.dequantize_rows(bank, dtype=DTYPES[out])
        assert torch.equal(got.cpu(), torch.from_numpy(y32).to(DTYPES[out]))
    # the stored value is within half a step of the row
    err = np.abs(ref.values(codes, scales, hd, group, fmt) - x.double().numpy())
    top = scales.astype(np.float64)[:, np.arange(hd) // group]
    step = np.maximum(np.abs(x.double().numpy()) / 8, top * 2.0 ** -9) if fmt == "fp8" else top
    assert (err <= step / 2 * (1 + 1e-3)).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("it", (torch.int32, torch.int64))
def test_rows_by_slot_and_stride(fmt, it):
    """Rows out of a wider tensor, to scattered slots; other slots stay; the read takes repeats."""
    n, hd, slots = 50, 72, 200
    wide = _rows(n, 90, 7).cuda()
    rows = wide[:, 5:5 + hd]
    at = torch.randperm(slots, generator=torch.Generator().manual_seed(1))[:n].to(it).cuda()
    bank, before = _bank(slots, hd, 32, fmt, seed=2)
    quant.quantize_rows(bank, rows, at)
    codes, scales = ref.quantise(rows.cpu().numpy(), 32, fmt)
    want = before.copy()
    want[at.cpu().numpy()] = ref.values(codes, scales, hd, 32, fmt)
    got = quant.dequantize_rows(bank, dtype=torch.float32).cpu().double().numpy()
    assert np.abs(got - want).max() <= EPS * np.abs(want).max()
    twice = torch.cat([at, at[:7]])
    out = torch.full((n + 7, hd + 3), 9.0, device="cuda")
    quant.dequantize_rows(bank, twice, out=out[:, 1:1 + hd])
    assert torch.equal(out[:, 1:1 + hd], quant.dequantize_rows(bank, dtype=torch.float32)[twice.long()])
    assert (out[:, 0] == 9).all() and (out[:, 1 + hd:] == 9).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_extreme_values(fmt):
    """Zeros, subnormals, the largest floats, infinities and NaN: each group by itself."""
    x = torch.zeros(8, 96)
    x[1, :32] = 1e-42
    x[2, 5] = 3.4e38
    x[3, 40] = float("inf")
    x[4, 70] = float("nan")
    x[5, 33] = -1.2e-30  # the smallest magnitudes that are kept are 2^-100 = 7.9e-31
    x[6] = torch.linspace(-1, 1, 96)
    x[7, 64:] = -0.0
    bank = quant.QuantBank.from_rows(x.cuda(), group=32, format=fmt)
    codes, scales = ref.quantise(x.numpy(), 32, fmt)
    assert np.array_equal(np.isnan(bank.scales.cpu().numpy()), np.isnan(scales))
    ok = ~np.isnan(scales)
    assert np.array_equal(bank.scales.cpu().numpy()[ok], scales[ok])
    got = quant.dequantize_rows(bank, dtype=torch.float32).cpu().numpy()
    assert np.isnan(got[3, 32:64]).all() and np.isnan(got[4, 64:]).all()
    assert not np.isnan(got[3, :32]).any() and not np.isnan(got[4, :64]).any()
    assert got[2, 5] == pytest.approx(3.4e38, rel=1e-6) and (got[1] == 0).all() and got[5, 33] != 0


def test_offsets_beyond_32_bits():
    """Slots whose codes lie past 4 GiB, and scales past 2^31 bytes."""
    n, hd = (1 << 24) + 5, 272
    bank = quant.QuantBank.zeros(n, hd, group=64)
    assert bank.codes.numel() > 1 << 32
    at = torch.tensor([n - 1, 3, 1 << 24, 15790321], device="cuda")
    rows = _rows(4, hd, 3).cuda()
    quant.quantize_rows(bank, rows, at)
    got = quant.dequantize_rows(bank, at, dtype=torch.float32)
    small = quant.QuantBank.from_rows(rows, group=64)
    assert torch.equal(got, quant.dequantize_rows(small, dtype=torch.float32))
    w = torch.ones(1, 4, device="cuda")
    out, = quant.gather(bank, [(at[None], w)])
    assert torch.allclose(out[0], got.sum(0), rtol=1e-5, atol=1e-5)
    dw, = quant.gather_dw(bank, [(at[None], torch.ones(1, hd, device="cuda"))])
    assert torch.allclose(dw[0], got.sum(1), rtol=1e-4, atol=1e-3 * got.abs().max().item())


def test_bad_slots_are_skipped_and_flagged():
    bank, before = _bank(20, 64, 32, "int8")
    at = torch.tensor([3, 20, -1, 7], device="cuda")
    quant.quantize_rows(bank, torch.ones(4, 64, device="cuda"), at)
    assert sdm.device_status() == sdm.SDM_DEV_BAD_INDEX
    got = quant.dequantize_rows(bank, at, dtype=torch.float32)
    assert sdm.device_status() == sdm.SDM_DEV_BAD_INDEX
    assert torch.allclose(got[[0, 3]], torch.ones(2, 64, device="cuda")) and (got[1:3] == 0).all()
    out, = quant.gather(bank, [(at[None], torch.ones(1, 4, device="cuda"))])
    assert sdm.device_status() == sdm.SDM_DEV_BAD_INDEX
    assert torch.allclose(out, torch.full_like(out, 2.0))
    dw, = quant.gather_dw(bank, [(at[None], torch.ones(1, 64, device="cuda"))])
    assert sdm.device_status() == sdm.SDM_DEV_BAD_INDEX
    assert torch.allclose(dw[0], torch.tensor([64.0, 0, 0, 64.0], device="cuda"))


# ---------------------------------------------------------------- gather and the weights' gradient

def _operands(bank64, tokens, widths, it, wdt, seed):
    gen = torch.Generator().manual_seed(seed)
    ops = []
    for w in widths:
        idx = torch.randint(0, len(bank64), (tokens, w), generator=gen).to(it)
        ops.append((idx, torch.randn((tokens, w), generator=gen).to(wdt)))
    return ops


GATHERS = [(1, 1, 32, (1,), 1, None), (7, 20, 32, (3,), 1, None), (40, 64, 64, (33, 5), 8, 5), (64, 128, 128, (64, 64), 64, 64),
           (30, 136, 64, (37,), 10, "chunks"), (12, 300, 128, (256, 1), 4, "chunks"), (6, 520, 32, (70,), 3, 0),
           (5000, 128, 128, (17,), 1, None), (4200, 48, 32, (40,), 1, None)]


def _chunk_args(tokens, chunk, valid):
    if valid == "chunks":
        cv = torch.randint(0, chunk + 1, (tokens // chunk,), generator=torch.Generator().manual_seed(4), dtype=torch.int32)
        live = (np.arange(tokens) % chunk) < cv.numpy()[np.arange(tokens) // chunk]
        return dict(chunk=chunk, chunk_valid=cv.cuda()), live
    live = (np.arange(tokens) % chunk) < (chunk if valid is None else valid)
    return dict(chunk=chunk, valid=valid), live


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tokens,hd,group,widths,chunk,valid", GATHERS)
def test_gather(fmt, tokens, hd, group, widths, chunk, valid):
    bank, rows = _bank(500, hd, group, fmt, seed=hd)
    it = torch.int32 if tokens % 2 else torch.int64
    wdt = torch.bfloat16 if hd % 8 else torch.float32
    ops = _operands(rows, tokens, widths, it, wdt, tokens)
    kw, live = _chunk_args(tokens, chunk, valid)
    outs = quant.gather(bank, [(i.cuda(), w.cuda()) for i, w in ops], **kw)
    for (idx, w), out in zip(ops, outs):
        terms = w.double().numpy()[..., None] * rows[idx.numpy()]
        want = terms.sum(1) * live[:, None]
        tol = (idx.shape[1] + 4) * EPS * np.abs(terms).sum(1)
        assert (np.abs(out.cpu().double().numpy() - want) <= tol).all()
        assert (out.cpu().numpy()[~live] == 0).all()


@pytest.mark.parametrize("fmt", FORMATS + ("bf16", "f32"))
@pytest.mark.parametrize("tokens,hd,group,widths,chunk,valid", GATHERS)
def test_gather_weight_gradient(fmt, tokens, hd, group, widths, chunk, valid):
    if fmt in DTYPES:
        bank = _rows(500, hd, hd, DTYPES[fmt]).cuda()
        rows = bank.cpu().double().numpy()
    else:
        bank, rows = _bank(500, hd, group, fmt, seed=hd)
    it = torch.int32 if tokens % 2 else torch.int64
    dt = torch.bfloat16 if widths[0] % 2 else torch.float32
    gen = torch.Generator().manual_seed(tokens)
    ops = [(idx, torch.randn((tokens, hd), generator=gen)) for idx, _ in _operands(rows, tokens, widths, it, dt, tokens)]
    kw, live = _chunk_args(tokens, chunk, valid)
    dws = quant.gather_dw(bank, [(i.cuda(), d.cuda()) for i, d in ops], dtype=dt, **kw)
    for (idx, d), dw in zip(ops, dws):
        terms = d.double().numpy()[:, None] * rows[idx.numpy()]
        want = terms.sum(2) * live[:, None]
        tol = (hd + 6) * EPS * np.abs(terms).sum(2)
        if dt == torch.bfloat16:
            tol = tol + 2.0 ** -8 * np.abs(want)
        assert (np.abs(dw.cpu().double().numpy() - want) <= tol).all()
        assert (dw.cpu().float().numpy()[~live] == 0).all()


def test_weight_gradient_against_differences():
    """d(sum dout out) / d w by central differences of the gather itself (linear, so exact but for
    rounding: 2 |out| (N + 4) eps over the step)."""
    bank, rows = _bank(100, 64, 32, "int8")
    (idx, w), = _operands(rows, 4, (9,), torch.int64, torch.float32, 0)
    idx, w = idx.cuda(), w.cuda()
    dout = torch.randn((4, 64), generator=torch.Generator().manual_seed(1)).cuda()
    dw, = quant.gather_dw(bank, [(idx, dout)])
    h = 0.5
    size = np.abs(rows[idx.cpu().numpy()]).sum(1).max() * (w.abs().max().item() + h)
    for n in range(9):
        e = torch.zeros_like(w)
        e[:, n] = h
        up, = quant.gather(bank, [(idx, w + e)])
        down, = quant.gather(bank, [(idx, w - e)])
        diff = ((up.double() - down.double()) * dout).sum(1) / (2 * h)
        assert (diff - dw[:, n]).abs().max().item() <= 2 * 20 * EPS * size * dout.abs().sum(1).max().item() / (2 * h)


def test_unaligned_banks_and_outputs():
    """A bf16 bank and float32 outputs that start off a 16-byte boundary."""
    big = _rows(301, 64, 1, torch.bfloat16).cuda().view(-1)
    bank = big[1:1 + 300 * 64].view(300, 64)
    rows = bank.cpu().double().numpy()
    (idx, _), = _operands(rows, 9, (21,), torch.int32, torch.float32, 3)
    flat = torch.randn(9 * 64 + 1, generator=torch.Generator().manual_seed(2)).cuda()
    dout = flat[1:].view(9, 64)
    dw, = quant.gather_dw(bank, [(idx.cuda(), dout)])
    terms = dout.cpu().double().numpy()[:, None] * rows[idx.numpy()]
    assert (np.abs(dw.cpu().double().numpy() - terms.sum(2)) <= 70 * EPS * np.abs(terms).sum(2)).all()
    qb, qrows = _bank(300, 64, 64, "fp8")
    out = torch.empty(9 * 64 + 1, device="cuda")[1:].view(9, 64)
    w = torch.randn((9, 21), generator=torch.Generator().manual_seed(5))
    quant.gather(qb, [(idx.cuda(), w.cuda())], outs=[out])
    terms = w.double().numpy()[..., None] * qrows[idx.numpy()]
    assert (np.abs(out.cpu().double().numpy() - terms.sum(1)) <= 25 * EPS * np.abs(terms).sum(1)).all()


# ---------------------------------------------------------------- decode

def _decode_inputs(S, P, hd, W, R, G, T, it, seed):
    gen = torch.Generator().manual_seed(seed)
    base = (torch.arange(S) * P).view(1, S, 1)
    k_idx = torch.stack([torch.stack([torch.randperm(P, generator=gen)[:W] for _ in range(S)]) for _ in range(T)])
    q_idx = torch.randint(0, P, (T, S, R), generator=gen)
    q_idx[..., : (R + 1) // 2] = k_idx[..., torch.arange((R + 1) // 2) % W]  # half of the reads see this token's writes
    k = torch.randn((T, S, W), generator=gen)
    return dict(k_idx=(k_idx + base).to(it), k_val=k / k.norm(dim=-1, keepdim=True), v=torch.randn((T, S, hd), generator=gen),
                beta=torch.rand((T, S), generator=gen), g=-torch.rand((T, S, G), generator=gen), q_idx=(q_idx + base).to(it),
                q_val=torch.randn((T, S, R), generator=gen) / 4)


DECODES = [(1, 8, 1, 32, 1, 1, 1, 1), (3, 40, 20, 32, 5, 3, 1, 3), (4, 64, 64, 64, 32, 32, 32, 2), (2, 300, 128, 128, 64, 64, 1, 3),
           (3, 100, 128, 64, 96, 17, 96, 2), (2, 300, 136, 64, 33, 70, 1, 2), (2, 300, 300, 128, 256, 256, 256, 2),
           (2, 300, 256, 32, 130, 9, 1, 2), (2, 300, 48, 32, 200, 256, 1, 2), (1, 70, 513, 128, 64, 64, 64, 2)]


@pytest.mark.parametrize("fmt", ("int8", "fp8"))
@pytest.mark.parametrize("S,P,hd,group,W,R,G,T", DECODES)
def test_decode(fmt, S, P, hd, group, W, R, G, T):
    """Token by token from the kernel's own state: new rows within half a step of their 64-bit
    values, untouched rows as they were, readings over the rows as written."""
    it = torch.int32 if S % 2 else torch.int64
    bank, state = _bank(S * P, hd, group, fmt, seed=3)
    x = _decode_inputs(S, P, hd, W, R, G, T, it, 5)
    for t in range(T):
        k_idx, q_idx = x["k_idx"][t].numpy(), x["q_idx"][t].numpy()
        k, v, beta = (x[n][t].double().numpy() for n in ("k_val", "v", "beta"))
        g = np.broadcast_to(x["g"][t].double().numpy(), (S, W))
        out = quant.decode_step(bank, *(x[n][t].cuda() for n in sdm.DecodeStepPlan.DECODE_KEYS),
                                out_dtype=torch.float32)
        row = state[k_idx] * np.exp(g)[..., None]
        kr = k[..., None] * row
        delta = beta[:, None] * (v - kr.sum(1))
        new = row + k[..., None] * delta[:, None]
        # float32: exp and products to 4 eps each, the sum to (W + 8) eps of its terms' size
        size = beta[:, None] * (np.abs(v) + np.abs(kr).sum(1))
        err32 = EPS * (8 * np.abs(row) + (W + 16) * np.abs(k)[..., None] * size[:, None])
        codes, scales = bank.codes.cpu().numpy(), bank.scales.cpu().numpy()
        after = ref.values(codes, scales, hd, group, fmt)
        top = scales.astype(np.float64)[k_idx][..., np.arange(hd) // group]
        step = np.maximum(np.abs(new) / 8, top * 2.0 ** -9) if fmt == "fp8" else top
        assert (np.abs(after[k_idx] - new) <= step / 2 * (1 + 1e-4) + 2 * err32).all()
        rest = np.ones(len(state), bool)
        rest[k_idx.reshape(-1)] = False
        assert np.array_equal(after[rest], state[rest])
        for gi in range(top.shape[-1] // group + 1):  # the scale is the group's largest value over the levels
            cols = slice(gi * group, min(hd, (gi + 1) * group))
            if cols.start < hd:
                big = np.abs(new[..., cols]).max(-1)
                tol = err32[..., cols].max(-1) + 2 * EPS * big
                assert (np.abs(scales[k_idx][..., gi] * ref.LEVELS[fmt] - big) <= 2 * tol).all()
        state = after
        terms = x["q_val"][t].double().numpy()[..., None] * state[q_idx]
        assert (np.abs(out.cpu().double().numpy() - terms.sum(1)) <= (R + 12) * EPS * np.abs(terms).sum(1)).all()


@pytest.mark.parametrize("fmt", ("int8", "fp8"))
@pytest.mark.parametrize("S,P,hd,group,W,R,G,T", [(3, 200, 128, 64, 64, 64, 1, 9), (2, 100, 136, 32, 40, 7, 40, 5)])
def test_decode_seq_is_the_steps(fmt, S, P, hd, group, W, R, G, T):
    x = {n: v.cuda() for n, v in _decode_inputs(S, P, hd, W, R, G, T, torch.int64, 6).items()}
    args = [x[n] for n in sdm.DecodeStepPlan.DECODE_KEYS]
    for out_dtype in (torch.bfloat16, torch.float32):
        banks = [_bank(S * P, hd, group, fmt, seed=4)[0] for _ in range(3)]
        steps = torch.stack([quant.decode_step(banks[0], *(a[t] for a in args), out_dtype=out_dtype) for t in range(T)])
        seq = quant.decode_seq(banks[1], *args, out_dtype=out_dtype)
        major = quant.decode_seq(banks[2], *(a.transpose(0, 1).contiguous() for a in args), out_dtype=out_dtype,
                                 stream_major=True)
        assert torch.equal(steps, seq) and torch.equal(seq, major.transpose(0, 1))
        for b in banks[1:]:
            assert torch.equal(b.codes, banks[0].codes) and torch.equal(b.scales, banks[0].scales)


def test_decay_alone_keeps_the_codes():
    """With k_val = 0 a row is only decayed: the codes stay, the scales carry it."""
    for fmt in ("int8", "fp8"):
        bank, _ = _bank(100, 128, 64, fmt)
        codes, scales = bank.codes.clone(), bank.scales.clone()
        idx = torch.arange(100, device="cuda").view(1, 100)
        z = torch.zeros(1, 100, device="cuda")
        for _ in range(10):
            quant.decode_step(bank, idx, z, torch.ones(1, 128, device="cuda"), torch.ones(1, device="cuda"),
                              torch.full((1, 1), -0.01, device="cuda"), idx, z)
        assert torch.equal(bank.codes, codes)
        assert torch.allclose(bank.scales, scales * float(np.exp(-0.1)), rtol=1e-5)


def test_decode_bad_slots():
    bank, state = _bank(10, 64, 32, "int8")
    idx = torch.tensor([[2, 10, -5]], device="cuda")
    one = torch.full((1, 3), 0.5, device="cuda")
    v = torch.ones(1, 64, device="cuda")
    out = quant.decode_step(bank, idx, one, v, torch.ones(1, device="cuda"), torch.zeros(1, 1, device="cuda"), idx, one,
                            out_dtype=torch.float32)
    assert sdm.device_status() == sdm.SDM_DEV_BAD_INDEX
    rows = ref.values(bank.codes.cpu().numpy(), bank.scales.cpu().numpy(), 64, 32, "int8")
    assert np.array_equal(np.delete(rows, 2, 0), np.delete(state, 2, 0))
    assert np.allclose(out.cpu().numpy()[0], rows[2] / 2, rtol=1e-6, atol=1e-6)


# ---------------------------------------------------------------- streams, empty calls, graphs

def test_other_streams_and_graphs():
    """Calls on a stream of their own, and captured in a graph, give the same results."""
    bank, _ = _bank(400, 128, 64, "int8", seed=8)
    x = {n: v.cuda() for n, v in _decode_inputs(4, 100, 128, 32, 32, 1, 1, torch.int64, 9).items()}
    args = [x[n][0] for n in sdm.DecodeStepPlan.DECODE_KEYS]
    idx, w = x["q_idx"][0], x["q_val"][0]
    copies = [quant.QuantBank(bank.codes.clone(), bank.scales.clone(), 128, group=64) for _ in range(2)]

    def work(b, stream=None):
        out = quant.decode_step(b, *args, stream=stream)
        sums, = quant.gather(b, [(idx, w)], stream=stream)
        return out, sums, quant.dequantize_rows(b, idx.view(-1), stream=stream)

    want = work(bank)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = work(copies[0], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work(copies[1])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_nothing_to_do():
    bank = quant.QuantBank.zeros(4, 64)
    none = torch.empty((0, 64), device="cuda")
    quant.quantize_rows(bank, none, torch.empty(0, dtype=torch.int64, device="cuda"))
    assert quant.dequantize_rows(bank, torch.empty(0, dtype=torch.int64, device="cuda")).shape == (0, 64)
    idx = torch.empty((0, 5), dtype=torch.int64, device="cuda")
    assert quant.gather(bank, [(idx, torch.empty((0, 5), device="cuda"))])[0].shape == (0, 64)
    assert quant.gather_dw(bank, [(idx, none)])[0].shape == (0, 5)
