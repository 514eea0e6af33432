"""A memory layer whose streams address a quantised bank by logits, from a prompt to training its reads.

    python examples/routed_memory.py

1. A prompt of 32 tokens for every stream in one decode call, then 8 single tokens: slots are chosen by
   logits over each stream's slots, written and read on int8 rows.
2. The read router, a linear map from 64 features to logits, is trained to read what another map reads:
   forward by ``read``, backward by ``read_backward``.
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

from decode_state_gb300 import quant, sdm  # noqa: E402
from decode_state_gb300.state import RoutedLayerState  # noqa: E402


def main(streams: int = 64, slots: int = 512, hd: int = 128, prompt: int = 32, tokens: int = 8, rounds: int = 40,
         format: str = "int8") -> dict:
    """Runs both parts; returns the readings of the single tokens and the losses of the training."""
    gen = torch.Generator(device="cuda").manual_seed(0)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    bank = quant.QuantBank.zeros(streams * slots, hd, group=64, format=format)
    state = RoutedLayerState(bank, streams, writes=32, reads=32)

    def inputs(*lead):
        return (randn(*lead, streams, slots), randn(*lead, streams, hd), torch.sigmoid(randn(*lead, streams)),
                -0.1 * torch.rand((*lead, streams, 1), generator=gen, device="cuda"), randn(*lead, streams, slots))

    state.steps(*inputs(prompt))
    readings = [state.step(*inputs()) for _ in range(tokens)]
    assert state.cache_len == prompt + tokens

    features = randn(streams, 64)
    target, _, _ = state.read(features @ randn(64, slots) / 4)
    router = 0.1 * randn(64, slots)
    losses = []
    for _ in range(rounds):
        logits = features @ router
        out, idx, w = state.read(logits)
        err = out - target
        losses.append(float((err * err).mean()))
        dlogits = state.read_backward(logits, idx, 2 * err, w)
        router -= 0.1 * (features.T @ dlogits)
    if sdm.device_status() != 0:
        raise RuntimeError("a kernel raised the device status word")
    return {"readings": readings, "losses": losses}


if __name__ == "__main__":
    result = main()
    print(f"last reading: {tuple(result['readings'][-1].shape)}, rms {result['readings'][-1].float().square().mean().sqrt():.4f}")
    print("loss " + " ".join(f"{x:.3e}" for x in result["losses"][::8] + result["losses"][-1:]))
