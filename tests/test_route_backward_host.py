"""Refusals of the routing gradient with the forward's weights, without a GPU."""

from __future__ import annotations

import pytest
from test_quant_host import BACKWARD, FAKE, codes, lib  # noqa: F401

EX = {**{k: v for k, v in list(BACKWARD.items())[:5]}, "w": FAKE, **dict(list(BACKWARD.items())[5:])}


@pytest.mark.parametrize("kw,code", [
    (dict(flags=2), "SDM_EFLAGS"), (dict(k=65), "SDM_EROUTE"), (dict(dlogits_stride=60), "SDM_ESTRIDE"), (dict(dw=None), "SDM_ENULL"),
    (dict(dlogits=None), "SDM_ENULL"), (dict(w=FAKE + 2), "SDM_EALIGN"), (dict(w=FAKE + 1, tokens=0), None), (dict(w=None, dw=None), "SDM_ENULL"),
    (dict(tokens=0, w=None), None),
])
def test_errors(lib, codes, kw, code):  # noqa: F811
    assert lib.sdm_route_backward_ex(*{**EX, **kw}.values(), None) == (codes[code] if code else 0)
