"""Outputs that overlap what a call reads, or one another, are refused before anything touches a GPU."""

from __future__ import annotations

import pytest
from test_quant_host import _gather_call, codes, lib  # noqa: F401

MB = 1 << 20
AT = [0x10000000 + i * 16 * MB for i in range(12)]  # never dereferenced: every call below is refused

ROWS = dict(codes=AT[0], scales=AT[1], n_slots=1000, hd=64, group=32, format=2, rows=AT[2], row_stride=80, row_dtype=1,
            slots=AT[3], idx_dtype=1, n_rows=100)


@pytest.mark.parametrize("kw", [
    dict(rows=AT[0] + 64), dict(rows=AT[0] + 1000 * 64 - 4), dict(rows=AT[0] - 99 * 320 - 252), dict(rows=AT[1] + 4 * 1999),
    dict(scales=AT[0] + 63996), dict(rows=AT[1] + 320 * 10 + 64 * 4), dict(rows=AT[0] - 320 * 3 + 16),
])
def test_rows(lib, codes, kw):  # noqa: F811
    for fn in (lib.sdm_quantize_rows, lib.sdm_dequantize_rows):
        assert fn(*{**ROWS, **kw}.values(), None) == codes["SDM_EOVERLAP"]


def test_rows_and_slots(lib, codes):  # noqa: F811
    for slots in (AT[0], AT[1] + 8000 - 8):
        assert lib.sdm_quantize_rows(*{**ROWS, "slots": slots}.values(), None) == codes["SDM_EOVERLAP"]
    for slots in (AT[2], AT[2] + 320 * 50, AT[2] + 320 * 50 + 248, AT[2] - 800 + 8, AT[2] + 320 * 99 + 248):
        assert lib.sdm_dequantize_rows(*{**ROWS, "slots": slots}.values(), None) == codes["SDM_EOVERLAP"]


def test_weight_gradient(lib, codes):  # noqa: F811
    scales = AT[0] + MB  # as in _gather_call: 100 rows of two groups
    assert _gather_call(lib.sdm_gather_dw, bank=AT[0], scales=scales, third=(scales + 796, AT[5])) == codes["SDM_EOVERLAP"]


DECODE = dict(codes=AT[0], scales=AT[1], n_slots=1000, k_idx=AT[2], k_val=AT[3], v=AT[4], beta=AT[5], g=AT[6], q_idx=AT[7],
              q_val=AT[8], out=AT[9], n_streams=4, hd=64, group=32, format=2, W=8, R=8, G=1, T=2, idx_dtype=1, out_dtype=0, flags=0)


@pytest.mark.parametrize("kw", [dict(out=AT[0] + 63998), dict(out=AT[1] + 7996), dict(scales=AT[0] + 32000)] +
                         [dict(out=DECODE[n] + 4) for n in ("k_idx", "k_val", "beta", "g", "q_idx", "q_val")] +
                         [dict(out=AT[4]), dict(out=AT[4] + 256, out_dtype=1), dict(out=AT[4] - 1022)] +
                         [{n: AT[0] + 32000} for n in ("k_idx", "k_val", "v", "beta", "g", "q_idx", "q_val")])
def test_decode(lib, codes, kw):  # noqa: F811
    assert lib.sdm_qdecode_seq(*{**DECODE, **kw}.values(), None) == codes["SDM_EOVERLAP"]


def test_decode_of_more_tokens_than_memory_holds(lib, codes):  # noqa: F811
    assert lib.sdm_qdecode_seq(*{**DECODE, "n_streams": 1 << 20, "T": (1 << 20) + 1}.values(), None) == codes["SDM_ECOUNT"]


ROUTE = dict(logits=AT[0], row_stride=80, logit_dtype=1, bias=AT[1], base=AT[2], idx=AT[3], w=AT[4], tokens=10, n=64, k=8, score=0,
             n_groups=1, top_groups=1, group_top=1, scale=1.0, flags=4, idx_dtype=1)


@pytest.mark.parametrize("kw", [dict(idx=AT[0]), dict(idx=AT[0] + 248), dict(w=AT[0] + 320 * 9 + 252), dict(w=AT[0] + 256),
                                dict(w=AT[0] - 316), dict(idx=AT[1] + 248), dict(w=AT[1] - 316), dict(idx=AT[2] + 72),
                                dict(w=AT[2]), dict(w=AT[3] + 636), dict(idx=AT[4] + 312)])
def test_route(lib, codes, kw):  # noqa: F811
    assert lib.sdm_route(*{**ROUTE, **kw}.values(), None) == codes["SDM_EOVERLAP"]


BACKWARD = dict(logits=AT[0], row_stride=80, logit_dtype=1, base=AT[1], idx=AT[2], w=AT[3], dw=AT[4], dlogits=AT[5], dlogits_stride=80,
                tokens=10, n=64, k=8, score=1, scale=1.0, flags=0, idx_dtype=1)


@pytest.mark.parametrize("kw", [
    dict(dlogits=AT[0]), dict(dlogits=AT[0] + 252), dict(dlogits=AT[0] - 252), dict(dlogits=AT[0] + 320 * 9), dict(dlogits=AT[0] - 320 * 9),
    dict(dlogits=AT[0] + 68), dict(dlogits=AT[0] + 320 * 4 - 68), dict(dlogits=AT[0] - 320 * 4 + 68), dict(dlogits=AT[0] + 256, dlogits_stride=81),
    dict(dlogits=AT[1] + 76), dict(dlogits=AT[2] + 636), dict(dlogits=AT[3] - 320), dict(dlogits=AT[4]), dict(dlogits=AT[4] - 9 * 320 - 252),
])
def test_route_backward(lib, codes, kw):  # noqa: F811
    assert lib.sdm_route_backward_ex(*{**BACKWARD, **kw}.values(), None) == codes["SDM_EOVERLAP"]
