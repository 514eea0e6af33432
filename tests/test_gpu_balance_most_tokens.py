"""The balance loss of as many tokens as a call may have: their number, and what is added to it on the way, beside 2^31.

The rows are all alike, so every row has the same part of the loss and of the gradient. Tolerances as in test_gpu_balance."""

from __future__ import annotations

import pytest
import torch

import train_reference as ref
from decode_state_gb300 import routing

pytestmark = pytest.mark.gpu

PARTS = 200.0


@pytest.mark.parametrize("tokens", ((1 << 31) - 1, 2145000000))
def test_most_tokens(tokens):
    x = torch.zeros((tokens, 2), dtype=torch.bfloat16, device="cuda")
    x[:, 1] = 1.0
    idx = torch.zeros((tokens, 1), dtype=torch.int32, device="cuda")
    idx[:3], idx[-8:] = 1, 1  # ends of the first and the last block's share
    want = torch.tensor([[tokens - 11, 11]])
    loss, counts, grad = routing.balance(x, idx, gradient=True)
    assert torch.equal(counts.cpu().long(), want)
    l64, g64, moved_l, moved_g = ref.balance(x[:1].cpu(), want, score="softmax")
    ref.close(loss, l64, moved_l, "loss", PARTS)
    for t in (0, tokens // 2, tokens - 1):  # a row's gradient is that of one token, shared by all
        ref.close(grad[t], g64[0] / tokens, moved_g[0] / tokens, f"row {t}", PARTS)
    # sequences: the last of few tokens, and tokens behind it
    del grad
    offsets = torch.tensor([0, tokens - 10, tokens - 2], dtype=torch.int32, device="cuda")
    want = torch.tensor([[tokens - 13, 3], [2, 6]])
    loss, counts = routing.balance(x, idx, offsets=offsets)
    assert torch.equal(counts.cpu().long(), want)
    for s in range(2):
        l64, _, moved_l, _ = ref.balance(x[:1].cpu(), want[s:s + 1], score="softmax")
        ref.close(loss[s:s + 1], l64, moved_l, f"loss {s}", PARTS)
