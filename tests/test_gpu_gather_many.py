"""Gathers and weight gradients of many tokens (the kernels that sum codes with limbs of the float32
factors), against 64-bit sums.

Tolerances, fixed before the first run:
  gather      (N + 4) eps sum_n |w row|: the product w * scale, its limbs (2^-32 of the largest of a
              step, far below its rounding), float32 accumulation and the join of the limbs
  gradient    (hd + 6) eps sum_c |dout row|, and one rounding to bfloat16 (2^-8 of the value); the limbs
              of dout are 2^-32 of the largest in a slice, so eps / 256 of |dout|_max sum_c |row| is added
"""

from __future__ import annotations

import pytest
import quant_reference as ref
import torch
from quant_reference import EPS

from decode_state_gb300 import quant, sdm

pytestmark = pytest.mark.gpu

FORMATS = ("int8", "fp8", "int4")
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
# tokens, hd, group, widths, chunk, valid
MANY = [(4096, 136, 64, (9,), 1, None), (2100, 300, 128, (40, 1), 7, "chunks"), (4096, 520, 32, (5,), 1, None),
        (4097, 16, 32, (33,), 17, 3), (4100, 1, 32, (2,), 1, None), (4200, 256, 64, (31,), 50, "chunks"),
        (4096, 64, 64, (32, 64), 64, 0), (4110, 200, 128, (16,), 30, "chunks"), (4096, 1032, 128, (3,), 1, None)]


@pytest.fixture(autouse=True)
def _clean_status():
    sdm.device_status()
    yield
    assert sdm.device_status() == 0


def _rows(n, hd, seed):
    gen = torch.Generator().manual_seed(seed)
    return torch.randn((n, hd), generator=gen) * torch.exp(2 * torch.randn((n, 1), generator=gen))


def _bank(n, hd, group, fmt, seed=0):
    """(a bank on the GPU, its float64 rows there)."""
    x = _rows(n, hd, seed)
    if fmt in DTYPES:
        bank = x.to(DTYPES[fmt]).cuda()
        return bank, bank.double()
    codes, scales = ref.quantise(x.numpy(), group, fmt)
    bank = quant.QuantBank(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), hd, group=group, format=fmt)
    return bank, torch.from_numpy(ref.values(codes, scales, hd, group, fmt)).cuda()


def _chunks(tokens, chunk, valid):
    """(keyword arguments, which tokens are live)."""
    at = torch.arange(tokens, device="cuda")
    if valid == "chunks":
        cv = torch.randint(-1, chunk + 2, (tokens // chunk,), generator=torch.Generator().manual_seed(4), dtype=torch.int32).cuda()
        return dict(chunk=chunk, chunk_valid=cv), at % chunk < cv[at // chunk]
    return dict(chunk=chunk, valid=valid), at % chunk < (chunk if valid is None else valid)


def _index(n, tokens, width, dtype, seed):
    return torch.randint(0, n, (tokens, width), generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def _randn(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def _check_gather(out, idx, w, rows, live):
    terms = w.double()[..., None] * rows[idx.long()]
    want = terms.sum(1) * live[:, None]
    assert bool(((out.double() - want).abs() <= (idx.shape[1] + 4) * EPS * terms.abs().sum(1)).all())
    assert bool((out[~live] == 0).all())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tokens,hd,group,widths,chunk,valid", MANY)
def test_gather(fmt, tokens, hd, group, widths, chunk, valid):
    bank, rows = _bank(500, hd, group, fmt, seed=hd)
    it = torch.int32 if tokens % 2 == 0 else torch.int64
    wdt = torch.bfloat16 if hd % 16 else torch.float32
    ops = [(_index(500, tokens, w, it, i), _randn((tokens, w), wdt, 10 + i)) for i, w in enumerate(widths)]
    kw, live = _chunks(tokens, chunk, valid)
    outs = [torch.full((tokens, hd), 7.0, device="cuda") for _ in ops]
    quant.gather(bank, ops, outs=outs, **kw)
    for (idx, w), out in zip(ops, outs):
        _check_gather(out, idx, w, rows, live)


@pytest.mark.parametrize("fmt", FORMATS + ("bf16", "f32"))
@pytest.mark.parametrize("tokens,hd,group,widths,chunk,valid", MANY)
def test_weight_gradient(fmt, tokens, hd, group, widths, chunk, valid):
    bank, rows = _bank(500, hd, group, fmt, seed=hd)
    it = torch.int32 if tokens % 2 else torch.int64
    dt = torch.bfloat16 if widths[0] % 2 else torch.float32
    ops = [(_index(500, tokens, w, it, i), _randn((tokens, hd), torch.float32, 10 + i)) for i, w in enumerate(widths)]
    kw, live = _chunks(tokens, chunk, valid)
    for (idx, d), dw in zip(ops, quant.gather_dw(bank, ops, dtype=dt, **kw)):
        r = rows[idx.long()]
        terms = d.double()[:, None] * r
        want = terms.sum(2) * live[:, None]
        tol = (hd + 6) * EPS * terms.abs().sum(2) + EPS / 256 * d.double().abs().amax(1)[:, None] * r.abs().sum(2)
        if dt == torch.bfloat16:
            tol = tol + 2.0 ** -8 * want.abs()
        assert bool(((dw.double() - want).abs() <= tol).all())
        assert bool((dw[~live] == 0).all())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("size", (1e30, 1e36, 1e-30))
def test_factors_near_the_ends_of_float32(fmt, size):
    """Weights and gradients whose exponents an f16 does not have; 1e36 times a row stays below 3e38."""
    codes, scales = ref.quantise((_rows(200, 128, 1).clamp(-30, 30) / 30).numpy(), 64, fmt)
    bank = quant.QuantBank(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), 128, group=64, format=fmt)
    rows = torch.from_numpy(ref.values(codes, scales, 128, 64, fmt)).cuda()
    idx = _index(200, 4096, 20, torch.int32, 2)
    live = torch.ones(4096, dtype=torch.bool, device="cuda")
    w = _randn((4096, 20), torch.float32, 3) * size
    out, = quant.gather(bank, [(idx, w)])
    if size > 1:
        _check_gather(out, idx, w, rows, live)
    else:  # products with a scale may be denormal, which a tolerance relative to them does not see
        terms = w.double()[..., None] * rows[idx.long()]
        assert bool(((out.double() - terms.sum(1)).abs() <= 24 * EPS * terms.abs().sum(1) + 20 * 448 * 2.0 ** -126).all())
    d = _randn((4096, 128), torch.float32, 4) * size
    dw, = quant.gather_dw(bank, [(idx, d)])
    r = rows[idx.long()]
    terms = d.double()[:, None] * r
    tol = 134 * EPS * terms.abs().sum(2) + EPS / 256 * d.double().abs().amax(1)[:, None] * r.abs().sum(2) + 128 * 2.0 ** -126
    assert bool(((dw.double() - terms.sum(2)).abs() <= tol).all())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("group", (32, 128))
def test_infinities_and_nans_stay_in_their_tokens(fmt, group):
    bank, rows = _bank(300, 128, group, fmt)
    idx = _index(300, 4096, 40, torch.int64, 0)
    w = _randn((4096, 40), torch.float32, 1)
    w[5, 7], w[9, 39], w[4000, 0] = float("inf"), float("-inf"), float("nan")
    out, = quant.gather(bank, [(idx, w)])
    want = (w.double()[..., None] * rows[idx.long()]).sum(1)
    assert torch.equal(out.isnan(), want.isnan())
    assert torch.equal(out.isinf(), want.isinf()) and torch.equal(out[out.isinf()].sign(), want[want.isinf()].sign().float())
    live = want.isfinite().all(1)
    assert live.sum() == 4093
    _check_gather(out[live], idx[live], w[live], rows, live[live])
    d = _randn((4096, 128), torch.float32, 2)
    d[11, 100], d[12, 0] = float("inf"), float("nan")
    dw, = quant.gather_dw(bank, [(idx, d)])
    want = (d.double()[:, None] * rows[idx.long()]).sum(2)
    assert torch.equal(dw.isnan(), want.isnan()) and torch.equal(dw.isinf(), want.isinf())


@pytest.mark.parametrize("fmt", FORMATS + ("bf16", "f32"))
def test_bad_slots_are_skipped_and_flagged(fmt):
    bank, rows = _bank(300, 64, 64, fmt)
    idx = _index(300, 5000, 33, torch.int64, 0)
    bad = torch.zeros(5000, 33, dtype=torch.bool, device="cuda")
    bad[3, 32], bad[100, 0], bad[4999, 5] = True, True, True
    broken = idx.clone()
    broken[bad] = torch.tensor([300, -1, 1 << 33], device="cuda")
    keep = torch.where(bad, 0.0, 1.0).double()
    d = _randn((5000, 64), torch.float32, 2)
    dw, = quant.gather_dw(bank, [(broken, d)])
    assert sdm.device_status() == sdm.SDM_DEV_BAD_INDEX
    assert bool((dw[bad] == 0).all())
    clean, = quant.gather_dw(bank, [(idx, d)])
    assert torch.equal(dw[~bad], clean[~bad])
    if fmt in FORMATS:
        w = _randn((5000, 33), torch.float32, 1)
        out, = quant.gather(bank, [(broken, w)])
        assert sdm.device_status() == sdm.SDM_DEV_BAD_INDEX
        _check_gather(out, idx, w.double() * keep, rows, torch.ones(5000, dtype=torch.bool, device="cuda"))


def test_same_results_on_every_call():
    """The same call twice is the same bits, and a token's result is that of its rows alone."""
    bank, _ = _bank(1000, 128, 128, "int8")
    idx, w = _index(1000, 9000, 64, torch.int32, 0), _randn((9000, 64), torch.bfloat16, 1)
    one, = quant.gather(bank, [(idx, w)])
    two, = quant.gather(bank, [(idx, w)])
    part, = quant.gather(bank, [(idx[4000:8500].contiguous(), w[4000:8500].contiguous())])
    assert torch.equal(one, two) and torch.equal(one[4000:8500], part)
