"""Groups with entries that a bias of +inf forces on, in more groups than stay: groups of equal infinite scores
go by the lower index, as all equal groups do. Choices are exact."""

from __future__ import annotations

import numpy as np
import pytest
import quant_reference as ref
import torch
from quant_reference import EPS

from decode_state_gb300 import routing

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ("softmax", "sigmoid"))
@pytest.mark.parametrize("group_top", (1, 2))
@pytest.mark.parametrize("n,k,groups,top_groups", [(64, 4, 8, 2), (256, 8, 8, 4), (256, 8, 8, 1), (512, 8, 16, 3), (1024, 32, 8, 2),
                                                   (250, 10, 5, 2), (2048, 16, 8, 3)])
def test_forced_entries_in_more_groups_than_stay(kind, group_top, n, k, groups, top_groups):
    per = n // groups
    gen = torch.Generator().manual_seed(n + groups)
    x = torch.randn((5, n), generator=gen)
    b = torch.zeros(n)
    for g in range(0, groups, 2 if top_groups < groups // 2 else 1):  # one forced entry in many groups, two in some
        b[g * per + int(torch.randint(per, (1,), generator=gen))] = float("inf")
    b[(groups - 1) * per] = b[groups * per - 1] = float("inf")
    kw = dict(bias=b, groups=groups, top_groups=top_groups, group_top=group_top)
    idx, w = routing.route(x.cuda(), k, score=kind, **{**kw, "bias": b.cuda()})
    want, ww = ref.route(x.numpy(), k, kind, **{**kw, "bias": b.numpy()})
    assert np.array_equal(idx.cpu().numpy(), want)
    assert (np.abs(w.cpu().double().numpy() - ww) <= 64 * EPS * ww).all()
