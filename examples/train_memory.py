"""Training a memory layer whose tokens read a bank by logits: embedding table, router and bank.

    python examples/train_memory.py

Tokens become rows of a table, a linear map turns them into logits over the bank's slots, the router takes the best and
the bank's rows are summed with its weights. ``gradients`` goes back through all of it: to the weights and the
bank's rows, through the router, whose balance loss is added on the way, to its map, and to the table.
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

from decode_state_gb300 import embedding, quant, routing, sdm  # noqa: E402

PADDING = 0  # the token that stands for nothing


def gradients(table, router, bank, tokens, target, *, reads: int, scale: float = 1.0, balance: float = 0.01, score: str = "softmax",
              offsets=None) -> dict:
    """One pass: the mean squared error of what ``tokens`` [T] read against ``target`` [T, hd], plus ``balance`` times the balance
    losses of the packed sequences that ``offsets`` cuts the tokens into, and the gradients of table [rows, d], router
    [d, slots] and bank [slots, hd] (float32)."""
    x = embedding.lookup(table, tokens, scale=scale, padding=PADDING)
    logits = x @ router
    idx, w = routing.route(logits, reads, score=score)
    (out,), _ = sdm.gather(bank, [(idx, w)], chunk=1, with_stash=False)
    err = out - target
    dout = err * (2 / err.numel())
    dw, = quant.gather_dw(bank, [(idx, dout)])
    dlogits = routing.route_backward(logits, idx, dw, score=score, w=w)
    balances, counts, dlogits = routing.balance(logits, idx, score=score, w=w, offsets=offsets, scale=balance, gradient=True, add=dlogits,
                                                out=dlogits)
    return {"loss": (err * err).mean() + balances.sum(), "balance": balances, "counts": counts, "idx": idx,
            "bank": quant.gather_drows([(idx, w, dout)], bank.shape[0]), "router": x.T @ dlogits,
            "table": embedding.backward(dlogits @ router.T, tokens, table.shape[0], scale=scale, padding=PADDING)}


def main(tokens: int = 1024, vocabulary: int = 5000, features: int = 64, slots: int = 512, hd: int = 128, reads: int = 16, rounds: int = 30) -> dict:
    """Trains on one batch; returns the losses and the last counts."""
    gen = torch.Generator(device="cuda").manual_seed(0)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    table, router, bank = randn(vocabulary, features) / 8, randn(features, slots) / 4, randn(slots, hd) / 4
    batch = torch.randint(0, vocabulary, (tokens,), generator=gen, device="cuda")
    target = randn(tokens, hd) / 4
    offsets = torch.tensor([0, tokens // 3, tokens], dtype=torch.int32, device="cuda")
    losses = []
    for _ in range(rounds):
        g = gradients(table, router, bank, batch, target, reads=reads, scale=8.0, offsets=offsets)
        losses.append(float(g["loss"]))
        for name, weights, rate in (("table", table, 1.0), ("router", router, 1.0), ("bank", bank, 100.0)):
            weights -= rate * g[name]
    if sdm.device_status() != 0:
        raise RuntimeError("a kernel raised the device status word")
    return {"losses": losses, "counts": g["counts"], "balance": g["balance"]}


if __name__ == "__main__":
    result = main()
    print("loss " + " ".join(f"{x:.4f}" for x in result["losses"][::6] + result["losses"][-1:]))
    print("balance losses", [round(float(x), 4) for x in result["balance"]], "most reads of a slot", int(result["counts"].max()))
