"""Refusals of the balance loss, the lookup and the gradients of rows that need no GPU: the C entry points return their
documented codes before they touch CUDA, and the Python functions raise on shapes and types."""

from __future__ import annotations

import ctypes
import re

import pytest
import torch

from decode_state_gb300 import build, embedding, quant, routing, sdm

FAKE = 0x10000000  # never dereferenced: every call below fails validation or has nothing to do
FAR = 1 << 28      # between the fake arrays


@pytest.fixture(scope="module")
def lib():
    build.build()
    return sdm.library()


@pytest.fixture(scope="module")
def codes():
    import os
    header = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "sdm.h")
    return {m.group(1): int(m.group(2)) for m in re.finditer(r"#define (SDM_E\w+) \((-\d+)\)", open(header).read())}


def _at(i):
    return FAKE + i * FAR


BALANCE = dict(logits=_at(0), row_stride=64, logit_dtype=1, base=_at(1), idx=_at(2), w=_at(3), offsets=_at(4), sequences=3, loss=_at(5),
               counts=_at(6), dloss=_at(7), add=_at(8), add_stride=64, dlogits=_at(9), dlogits_stride=64, tokens=10, n=64, k=8, score=0,
               scale=1.0, idx_dtype=1, workspace=_at(10), workspace_bytes=1 << 20)


@pytest.mark.parametrize("kw,code", [
    (dict(logit_dtype=2), "SDM_EDTYPE"), (dict(idx_dtype=2), "SDM_EIDX"), (dict(n=0), "SDM_EROUTE"), (dict(n=65537), "SDM_EROUTE"),
    (dict(k=0), "SDM_EROUTE"), (dict(k=65), "SDM_EROUTE"), (dict(k=257, n=1000), "SDM_EROUTE"), (dict(score=2), "SDM_EROUTE"),
    (dict(tokens=-1), "SDM_ECOUNT"), (dict(tokens=1 << 31), "SDM_ECOUNT"), (dict(tokens=1 << 28), "SDM_ECOUNT"),
    (dict(sequences=-1), "SDM_ECOUNT"), (dict(sequences=1 << 24), "SDM_ECOUNT"), (dict(offsets=None), "SDM_ECOUNT"),
    (dict(offsets=None, sequences=0), "SDM_ECOUNT"), (dict(loss=None), "SDM_ENULL"), (dict(counts=None), "SDM_ENULL"),
    (dict(logits=None), "SDM_ENULL"), (dict(idx=None), "SDM_ENULL"), (dict(workspace=None), "SDM_ENULL"),
    (dict(row_stride=63), "SDM_ESTRIDE"), (dict(add_stride=63), "SDM_ESTRIDE"), (dict(dlogits_stride=10), "SDM_ESTRIDE"),
    (dict(logits=_at(0) + 2), "SDM_EALIGN"), (dict(idx=_at(2) + 4), "SDM_EALIGN"), (dict(base=_at(1) + 4), "SDM_EALIGN"),
    (dict(w=_at(3) + 1), "SDM_EALIGN"), (dict(offsets=_at(4) + 2), "SDM_EALIGN"), (dict(loss=_at(5) + 2), "SDM_EALIGN"),
    (dict(counts=_at(6) + 1), "SDM_EALIGN"), (dict(dloss=_at(7) + 3), "SDM_EALIGN"), (dict(add=_at(8) + 2), "SDM_EALIGN"),
    (dict(dlogits=_at(9) + 2), "SDM_EALIGN"), (dict(workspace=_at(10) + 16), "SDM_EALIGN"), (dict(workspace_bytes=1000), "SDM_EWORKSPACE"),
    (dict(dlogits=_at(0)), "SDM_EOVERLAP"), (dict(counts=_at(0) + 256), "SDM_EOVERLAP"), (dict(loss=_at(4) + 4), "SDM_EOVERLAP"),
    (dict(dlogits=_at(8), dlogits_stride=80), "SDM_EOVERLAP"), (dict(add=_at(9) + 4), "SDM_EOVERLAP"), (dict(counts=_at(5)), "SDM_EOVERLAP"),
    (dict(workspace=_at(2)), "SDM_EOVERLAP"), (dict(dlogits=_at(10)), "SDM_EOVERLAP"), (dict(dloss=_at(6) + 8), "SDM_EOVERLAP"),
    (dict(tokens=0, sequences=0), None),
])
def test_balance_errors(lib, codes, kw, code):
    assert lib.sdm_balance(*{**BALANCE, **kw}.values(), None) == (codes[code] if code else 0)


LOOKUP = dict(table=_at(0), n_rows=100, hd=64, table_dtype=0, tokens=_at(1), idx_dtype=1, n_tokens=10, padding=-1, scale=1.0, out=_at(2),
              out_dtype=1)


@pytest.mark.parametrize("kw,code", [
    (dict(table_dtype=2), "SDM_EDTYPE"), (dict(out_dtype=3), "SDM_EDTYPE"), (dict(idx_dtype=2), "SDM_EIDX"), (dict(hd=0), "SDM_EHD"),
    (dict(hd=65537), "SDM_EHD"), (dict(n_rows=0), "SDM_ECOUNT"), (dict(n_rows=1 << 31), "SDM_ECOUNT"), (dict(n_tokens=-1), "SDM_ECOUNT"),
    (dict(table=None), "SDM_ENULL"), (dict(tokens=None), "SDM_ENULL"), (dict(out=None), "SDM_ENULL"), (dict(table=_at(0) + 1), "SDM_EALIGN"),
    (dict(tokens=_at(1) + 4), "SDM_EALIGN"), (dict(out=_at(2) + 2), "SDM_EALIGN"), (dict(out=_at(0) + 128), "SDM_EOVERLAP"),
    (dict(out=_at(1)), "SDM_EOVERLAP"), (dict(n_tokens=0, table=None), None),
])
def test_lookup_errors(lib, codes, kw, code):
    assert lib.sdm_lookup(*{**LOOKUP, **kw}.values(), None) == (codes[code] if code else 0)


BACKWARD = dict(dout=_at(0), dout_dtype=0, tokens=_at(1), idx_dtype=1, n_tokens=1000, padding=-1, scale=1.0, grad=_at(2), n_rows=100,
                hd=64, grad_dtype=1, flags=0, workspace=_at(3), workspace_bytes=1 << 24)


@pytest.mark.parametrize("kw,code", [
    (dict(flags=1), "SDM_EFLAGS"), (dict(dout_dtype=2), "SDM_EDTYPE"), (dict(grad_dtype=-1), "SDM_EDTYPE"), (dict(idx_dtype=7), "SDM_EIDX"),
    (dict(hd=0), "SDM_EHD"), (dict(n_rows=0), "SDM_ECOUNT"), (dict(n_tokens=1 << 31), "SDM_ECOUNT"), (dict(n_tokens=-5), "SDM_ECOUNT"),
    (dict(grad=None), "SDM_ENULL"), (dict(dout=None), "SDM_ENULL"), (dict(tokens=None), "SDM_ENULL"), (dict(workspace=None), "SDM_ENULL"),
    (dict(dout=_at(0) + 1), "SDM_EALIGN"), (dict(tokens=_at(1) + 2), "SDM_EALIGN"), (dict(grad=_at(2) + 2), "SDM_EALIGN"),
    (dict(workspace=_at(3) + 128), "SDM_EALIGN"), (dict(workspace_bytes=64), "SDM_EWORKSPACE"), (dict(grad=_at(0)), "SDM_EOVERLAP"),
    (dict(grad=_at(1) + 8), "SDM_EOVERLAP"), (dict(workspace=_at(2)), "SDM_EOVERLAP"), (dict(workspace=_at(0)), "SDM_EOVERLAP"),
    (dict(n_tokens=0, flags=8, grad=None), None),
])
def test_lookup_backward_errors(lib, codes, kw, code):
    assert lib.sdm_lookup_backward(*{**BACKWARD, **kw}.values(), None) == (codes[code] if code else 0)


def _drows(lib, **kw):
    a = dict(n_ops=2, idx=(_at(0), _at(1)), w=(_at(2), _at(3)), dout=(_at(4), _at(5)), width=(8, 4), idx_dtype=1, w_dtype=1, drows=_at(6),
             n_slots=100, hd=64, drows_dtype=1, flags=0, tokens=600, chunk=3, valid=2, chunk_valid=None, workspace=_at(7),
             workspace_bytes=1 << 24)
    a.update(kw)
    for n in ("idx", "w", "dout"):
        a[n] = None if a[n] is None else (ctypes.c_void_p * 2)(*a[n])
    a["width"] = None if a["width"] is None else (ctypes.c_int * 2)(*a["width"])
    return lib.sdm_gather_drows(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(flags=2), "SDM_EFLAGS"), (dict(w_dtype=2), "SDM_EDTYPE"), (dict(drows_dtype=2), "SDM_EDTYPE"), (dict(idx_dtype=2), "SDM_EIDX"),
    (dict(n_ops=0), "SDM_ENOPS"), (dict(n_ops=3), "SDM_ENOPS"), (dict(idx=None), "SDM_ENULL"), (dict(w=None), "SDM_ENULL"),
    (dict(dout=None), "SDM_ENULL"), (dict(width=None), "SDM_ENULL"), (dict(width=(0, 4)), "SDM_EWIDTH"), (dict(width=(8, 257)), "SDM_EWIDTH"),
    (dict(tokens=-3), "SDM_ECOUNT"), (dict(tokens=3 << 27), "SDM_ECOUNT"), (dict(n_slots=0), "SDM_ECOUNT"), (dict(hd=0), "SDM_EHD"),
    (dict(chunk=0), "SDM_ECHUNK"), (dict(chunk=7), "SDM_ECHUNK"), (dict(valid=4), "SDM_ECHUNK"), (dict(valid=-1), "SDM_ECHUNK"),
    (dict(drows=None), "SDM_ENULL"), (dict(idx=(None, _at(1))), "SDM_ENULL"), (dict(dout=(_at(4), None)), "SDM_ENULL"),
    (dict(drows=_at(6) + 2), "SDM_EALIGN"), (dict(w=(_at(2) + 2, _at(3))), "SDM_EALIGN"), (dict(chunk_valid=_at(8) + 1), "SDM_EALIGN"),
    (dict(workspace=_at(7) + 4), "SDM_EALIGN"), (dict(workspace=None), "SDM_ENULL"), (dict(workspace_bytes=0), "SDM_EWORKSPACE"),
    (dict(drows=_at(5)), "SDM_EOVERLAP"), (dict(drows=_at(1)), "SDM_EOVERLAP"), (dict(workspace=_at(3)), "SDM_EOVERLAP"),
    (dict(chunk_valid=_at(6) + 16), "SDM_EOVERLAP"), (dict(tokens=0, flags=8, drows=None), None),
])
def test_gather_drows_errors(lib, codes, kw, code):
    assert _drows(lib, **kw) == (codes[code] if code else 0)


def test_workspaces(lib, codes):
    """Sizes grow with the work, are whole words, and bad sizes are refused."""
    size = ctypes.c_int64(-1)

    def ask(fn, *args):
        rc = fn(*args, ctypes.byref(size))
        return rc, size.value

    assert ask(lib.sdm_balance_workspace, 0)[0] == 0 and ask(lib.sdm_balance_workspace, 1000)[1] > ask(lib.sdm_balance_workspace, 1)[1] > 0
    assert ask(lib.sdm_balance_workspace, -1) == (codes["SDM_ECOUNT"], 0)
    assert lib.sdm_balance_workspace(1, None) == codes["SDM_ENULL"]
    for fn in (lib.sdm_lookup_backward_workspace, lib.sdm_gather_drows_workspace):
        assert ask(fn, 0, 10, 64) == (0, 0)
        sizes = [ask(fn, e, 10, 64)[1] for e in (1000, 20000, 1 << 20, (1 << 31) - 1)]
        assert sizes == sorted(sizes) and sizes[0] > 0 and all(s % 4 == 0 for s in sizes)
        assert ask(fn, 1 << 31, 10, 64) == (codes["SDM_ECOUNT"], 0) and ask(fn, 5, 0, 64) == (codes["SDM_ECOUNT"], 0)
        assert ask(fn, 5, 10, 0) == (codes["SDM_EHD"], 0) and fn(5, 10, 64, None) == codes["SDM_ENULL"]


def test_python_refusals():
    x, idx = torch.zeros(3, 8), torch.zeros(3, 2, dtype=torch.int64)
    for call in (lambda: routing.balance(x, idx), lambda: embedding.lookup(x, idx), lambda: embedding.backward(x, idx[:, 0], 5),
                 lambda: quant.gather_drows([(idx, x[:, :2], x)], 5)):
        with pytest.raises(ValueError):  # not on a GPU
            call()
    with pytest.raises(ValueError):
        routing.balance(x, idx, score="entropy")
    with pytest.raises(TypeError):
        routing.balance(x.double(), idx)
    with pytest.raises(TypeError):
        embedding.lookup(x, idx.to(torch.int16))
    with pytest.raises(TypeError):
        embedding.backward(x.half(), idx[:, 0], 5)
    with pytest.raises(TypeError):
        quant.gather_drows([idx, x], 5)
    with pytest.raises(ValueError):
        quant.gather_drows([(idx, x)], 5)
    with pytest.raises(ValueError):
        quant.gather_drows([], 5)
