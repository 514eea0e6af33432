"""Refusals of the quantised banks and the routing that need no GPU: the C entry points return their
documented codes before they touch CUDA, and the Python functions raise on shapes and types."""

from __future__ import annotations

import ctypes
import re

import pytest
import torch

from decode_state_gb300 import build, quant, routing, sdm

FAKE = 0x10000000  # never dereferenced: every call below fails validation or has nothing to do


@pytest.fixture(scope="module")
def lib():
    build.build()
    return sdm.library()


@pytest.fixture(scope="module")
def codes():
    import os
    header = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "sdm.h")
    return {m.group(1): int(m.group(2)) for m in re.finditer(r"#define (SDM_E\w+) \((-\d+)\)", open(header).read())}


def test_row_bytes(lib):
    for hd in (1, 15, 16, 17, 31, 32, 33, 128, 300, 65536):
        for fmt, code in quant.FORMATS.items():
            b = lib.sdm_quant_row_bytes(hd, code)
            assert b == quant.row_bytes(hd, fmt) and b % 16 == 0
            assert b - 16 < (hd if fmt != "int4" else (hd + 1) // 2) <= b
    assert lib.sdm_quant_row_bytes(0, 2) == lib.sdm_quant_row_bytes(65537, 2) == lib.sdm_quant_row_bytes(64, 1) == 0


ROWS = dict(codes=FAKE, scales=FAKE, n_slots=10, hd=64, group=32, format=2, rows=FAKE, row_stride=64, row_dtype=0,
            slots=FAKE, idx_dtype=1, n_rows=4)


@pytest.mark.parametrize("kw,code", [
    (dict(format=0), "SDM_EFORMAT"), (dict(format=5), "SDM_EFORMAT"), (dict(hd=0), "SDM_EHD"), (dict(hd=70000), "SDM_EHD"),
    (dict(group=16), "SDM_EGROUP"), (dict(group=0), "SDM_EGROUP"), (dict(group=256), "SDM_EGROUP"),
    (dict(n_slots=0), "SDM_ECOUNT"), (dict(n_slots=1 << 31), "SDM_ECOUNT"), (dict(n_rows=-1), "SDM_ECOUNT"),
    (dict(row_dtype=2), "SDM_EDTYPE"), (dict(idx_dtype=2), "SDM_EIDX"), (dict(slots=None, n_rows=11), "SDM_EROW"),
    (dict(codes=None), "SDM_ENULL"), (dict(scales=None), "SDM_ENULL"), (dict(rows=None), "SDM_ENULL"),
    (dict(row_stride=63), "SDM_ESTRIDE"), (dict(codes=FAKE + 8), "SDM_EALIGN"), (dict(scales=FAKE + 2), "SDM_EALIGN"),
    (dict(rows=FAKE + 1), "SDM_EALIGN"), (dict(slots=FAKE + 4), "SDM_EALIGN"), (dict(n_rows=0, rows=None), None),
])
def test_rows_errors(lib, codes, kw, code):
    a = {**ROWS, **kw}
    for fn in (lib.sdm_quantize_rows, lib.sdm_dequantize_rows):
        assert fn(*a.values(), None) == (codes[code] if code else 0)


def _pair(*v):
    return (ctypes.c_void_p * 2)(*v)


def _gather_call(fn, **kw):
    far = FAKE + (1 << 24)
    a = dict(bank=FAKE, scales=FAKE + (1 << 20), n_slots=100, hd=64, group=32, format=2, n_ops=2, idx=(far, far),
             second=(far, far), third=(far, far), width=(8, 4), idx_dtype=1, w_dtype=1, tokens=6, chunk=3, valid=2,
             chunk_valid=None)
    a.update(kw)
    for n in ("idx", "second", "third"):
        a[n] = None if a[n] is None else _pair(*a[n])
    a["width"] = (ctypes.c_int * 2)(*a["width"])
    if fn is sdm.library().sdm_gather_dw and kw.get("format") == 0:
        a["scales"] = None
    return fn(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(format=7), "SDM_EFORMAT"), (dict(hd=0), "SDM_EHD"), (dict(group=48), "SDM_EGROUP"), (dict(n_slots=0), "SDM_ECOUNT"),
    (dict(w_dtype=3), "SDM_EDTYPE"), (dict(idx_dtype=3), "SDM_EIDX"), (dict(n_ops=3), "SDM_ENOPS"), (dict(n_ops=0), "SDM_ENOPS"),
    (dict(idx=None), "SDM_ENULL"), (dict(width=(0, 4)), "SDM_EWIDTH"), (dict(width=(8, 257)), "SDM_EWIDTH"),
    (dict(tokens=-3), "SDM_ECOUNT"), (dict(chunk=0), "SDM_ECHUNK"), (dict(chunk=4), "SDM_ECHUNK"), (dict(valid=4), "SDM_ECHUNK"),
    (dict(valid=-1), "SDM_ECHUNK"), (dict(bank=None), "SDM_ENULL"), (dict(scales=None), "SDM_ENULL"),
    (dict(bank=FAKE + 4), "SDM_EALIGN"), (dict(idx=(FAKE + 4, FAKE)), "SDM_EALIGN"), (dict(second=(0, FAKE)), "SDM_ENULL"),
    (dict(third=(FAKE + 64, FAKE + (1 << 24))), "SDM_EOVERLAP"), (dict(tokens=0), None),
])
def test_gather_errors(lib, codes, kw, code):
    for fn in (lib.sdm_qgather, lib.sdm_gather_dw):
        assert _gather_call(fn, **kw) == (codes[code] if code else 0)


def test_weight_gradient_takes_plain_banks(lib, codes):
    """Formats of the unquantised banks: no scales and no group are asked for."""
    assert _gather_call(lib.sdm_gather_dw, format=0, group=0, tokens=0) == 0
    assert _gather_call(lib.sdm_qgather, format=0) == codes["SDM_EFORMAT"]
    assert _gather_call(lib.sdm_gather_dw, format=0, bank=FAKE + 1) == codes["SDM_EALIGN"]


DECODE = dict(codes=FAKE, scales=FAKE, n_slots=100, k_idx=FAKE, k_val=FAKE, v=FAKE, beta=FAKE, g=FAKE, q_idx=FAKE, q_val=FAKE,
              out=FAKE, n_streams=4, hd=64, group=32, format=2, W=8, R=8, G=1, T=2, idx_dtype=1, out_dtype=0, flags=0)


@pytest.mark.parametrize("kw,code", [
    (dict(flags=1), "SDM_EFLAGS"), (dict(flags=4), "SDM_EFLAGS"), (dict(format=4), "SDM_EFORMAT"), (dict(format=0), "SDM_EFORMAT"),
    (dict(hd=0), "SDM_EHD"), (dict(group=8), "SDM_EGROUP"), (dict(n_slots=-1), "SDM_ECOUNT"), (dict(out_dtype=4), "SDM_EDTYPE"),
    (dict(idx_dtype=4), "SDM_EIDX"), (dict(W=0), "SDM_EWIDTH"), (dict(R=257), "SDM_EWIDTH"), (dict(G=2), "SDM_EGATES"),
    (dict(n_streams=-1), "SDM_ECOUNT"), (dict(T=-1), "SDM_ECOUNT"), (dict(beta=None), "SDM_ENULL"), (dict(codes=FAKE + 8), "SDM_EALIGN"),
    (dict(q_idx=FAKE + 4), "SDM_EALIGN"), (dict(out=FAKE + 1), "SDM_EALIGN"), (dict(T=0, k_idx=None), None), (dict(n_streams=0), None),
    (dict(flags=2, T=0), None),
])
def test_decode_errors(lib, codes, kw, code):
    want = codes[code] if code else 0
    assert lib.sdm_qdecode_seq(*{**DECODE, **kw}.values(), None) == want
    if "T" not in kw and "flags" not in kw:
        step = {k: v for k, v in {**DECODE, **kw}.items() if k not in ("T", "flags")}
        assert lib.sdm_qdecode_step(*step.values(), None) == want


ROUTE = dict(logits=FAKE, row_stride=64, logit_dtype=1, bias=None, base=None, idx=FAKE, w=FAKE, tokens=4, n=64, k=8, score=0,
             n_groups=1, top_groups=1, group_top=1, scale=1.0, flags=4, idx_dtype=0)


@pytest.mark.parametrize("kw,code", [
    (dict(flags=1), "SDM_EFLAGS"), (dict(flags=8), "SDM_EFLAGS"), (dict(logit_dtype=2), "SDM_EDTYPE"), (dict(idx_dtype=2), "SDM_EIDX"),
    (dict(n=0), "SDM_EROUTE"), (dict(n=65537), "SDM_EROUTE"), (dict(k=0), "SDM_EROUTE"), (dict(k=65), "SDM_EROUTE"),
    (dict(n=1000, row_stride=1000, k=257), "SDM_EROUTE"), (dict(score=2), "SDM_EROUTE"), (dict(n_groups=0), "SDM_EROUTE"),
    (dict(n_groups=7), "SDM_EROUTE"), (dict(n_groups=8, top_groups=9), "SDM_EROUTE"), (dict(top_groups=0), "SDM_EROUTE"),
    (dict(group_top=3), "SDM_EROUTE"), (dict(tokens=-1), "SDM_ECOUNT"), (dict(row_stride=63), "SDM_ESTRIDE"),
    (dict(logits=None), "SDM_ENULL"), (dict(idx=None), "SDM_ENULL"), (dict(w=None), "SDM_ENULL"), (dict(logits=FAKE + 2), "SDM_EALIGN"),
    (dict(bias=FAKE + 2), "SDM_EALIGN"), (dict(base=FAKE + 2), "SDM_EALIGN"), (dict(w=FAKE + 1), "SDM_EALIGN"),
    (dict(tokens=0, logits=None), None),
])
def test_route_errors(lib, codes, kw, code):
    assert lib.sdm_route(*{**ROUTE, **kw}.values(), None) == (codes[code] if code else 0)


BACKWARD = dict(logits=FAKE, row_stride=64, logit_dtype=0, base=None, idx=FAKE, dw=FAKE, dlogits=FAKE, dlogits_stride=64, tokens=4,
                n=64, k=8, score=1, scale=1.0, flags=0, idx_dtype=1)


@pytest.mark.parametrize("kw,code", [
    (dict(flags=2), "SDM_EFLAGS"), (dict(k=65), "SDM_EROUTE"), (dict(score=-1), "SDM_EROUTE"), (dict(dlogits_stride=60), "SDM_ESTRIDE"),
    (dict(row_stride=0), "SDM_ESTRIDE"), (dict(dw=None), "SDM_ENULL"), (dict(dlogits=None), "SDM_ENULL"), (dict(dw=FAKE + 2), "SDM_EALIGN"),
    (dict(dlogits=FAKE + 1), "SDM_EALIGN"), (dict(tokens=0, dw=None), None),
])
def test_route_backward_errors(lib, codes, kw, code):
    assert lib.sdm_route_backward(*{**BACKWARD, **kw}.values(), None) == (codes[code] if code else 0)


def test_python_refusals():
    codes, scales = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 2)
    for bad, kw in ((ValueError, dict(format="int2")), (ValueError, dict(group=16)), (ValueError, dict(group=64)),
                    (ValueError, dict(format="int4", group=32))):
        with pytest.raises(bad):
            quant.QuantBank(codes, scales, 64, **{"group": 32, **kw})
    with pytest.raises(TypeError):
        quant.QuantBank(codes.to(torch.int8), scales, 64, group=32)
    with pytest.raises(ValueError):  # not on a GPU
        quant.QuantBank(codes, scales, 64, group=32)
    x = torch.zeros(3, 8)
    for call in (lambda: routing.route(x, 2), lambda: routing.route_backward(x, torch.zeros(3, 2, dtype=torch.int64), torch.zeros(3, 2))):
        with pytest.raises(ValueError):
            call()
