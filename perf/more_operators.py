"""The operators that train a routed memory layer: what is measured, on which inputs, and their plain forms.

Four operators, beside the routing, the gather and the gradient of its weights:
  balance    the balance loss of a router with the counts of its entries, and the gradient of its logits
  lookup     scaled rows of an embedding table
  embedding  the gradient of that table: the rows' gradients summed by token
  rows       the gradient of the bank's rows in a gather: weighted sums of the readings' gradients by slot

``own`` chooses between the framework's kernels and plain forms in elementary float32 operations.
"""

from __future__ import annotations

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
INDEX = {"i32": torch.int32, "i64": torch.int64}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the usage of a step's router over 64 streams, as a serving loop watches it; latency counts
        dict(name="balance step", kind="balance", tokens=64, n=256, k=8, dtype="bf16", score="sigmoid", sequences=1,
             masked=0.0, filled=False, base=False, gradient=False, add=False, idx="i32"),
        # a training batch of packed sequences: every sequence balanced by itself, the gradient added to the router's own
        dict(name="balance batch", kind="balance", tokens=65536, n=256, k=8, dtype="bf16", score="sigmoid", sequences=37,
             masked=0.0, filled=False, base=False, gradient=True, add=True, idx="i32"),
        # 1024 streams that each choose 64 of their own 16384 slots, a quarter not in use yet
        dict(name="balance slots", kind="balance", tokens=1024, n=16384, k=64, dtype="f32", score="softmax", sequences=1,
             masked=0.25, filled=False, base=True, gradient=False, add=False, idx="i32"),
        # a router of ragged size, some of whose chosen entries only filled up
        dict(name="balance ragged", kind="balance", tokens=4097, n=4099, k=33, dtype="f32", score="softmax", sequences=3,
             masked=0.02, filled=True, base=False, gradient=True, add=False, idx="i64"),
        # the tokens of one decoding step
        dict(name="lookup step", kind="lookup", tokens=64, rows=32768, hd=1024, dtype="bf16", out="bf16", idx="i64"),
        # the tokens of a training batch, a few of them padding
        dict(name="lookup batch", kind="lookup", tokens=65536, rows=131072, hd=2048, dtype="bf16", out="bf16", idx="i32"),
        # a small batch into a gradient that is kept: only the rows of its tokens are touched
        dict(name="embedding step", kind="embedding", tokens=512, rows=32768, hd=1024, dtype="bf16", out="f32",
             accumulate=True, idx="i64"),
        # odd sizes, a table in half the bits
        dict(name="embedding ragged", kind="embedding", tokens=5001, rows=4099, hd=264, dtype="f32", out="bf16",
             accumulate=False, idx="i32"),
        # the gradient of the table in a training batch; a few tokens make up much of it
        dict(name="embedding batch", kind="embedding", tokens=65536, rows=131072, hd=2048, dtype="bf16", out="f32",
             accumulate=False, idx="i64"),
        # the bank's gradient of one slab of 256 readings
        dict(name="rows slab", kind="rows", tokens=256, n_slots=65536, hd=128, width0=64, width1=0, chunk=1, ragged=False,
             wdtype="f32", out="f32", accumulate=True, skewed=False, idx="i32"),
        # rows and widths of odd sizes, two operands
        dict(name="rows ragged", kind="rows", tokens=1000, n_slots=100003, hd=264, width0=37, width1=5, chunk=8, ragged=True,
             wdtype="bf16", out="bf16", accumulate=False, skewed=True, idx="i64"),
        # the bank's gradient of the gather's workload: chunks with padding, two operands
        dict(name="rows batch", kind="rows", tokens=65536, n_slots=1 << 20, hd=128, width0=64, width1=32, chunk=64,
             ragged=True, wdtype="bf16", out="f32", accumulate=False, skewed=False, idx="i64"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["balance", "balance", "lookup", "embedding", "rows"])
    idx, dtype, out = rng.choice(["i32", "i64"]), rng.choice(["bf16", "f32"]), rng.choice(["bf16", "f32"])
    if kind == "balance":
        n = _log(rng, 8, 16384)
        tokens = _log(rng, 8, min(65536, (1 << 24) // n))
        gradient = rng.random() < 0.5
        return dict(kind=kind, tokens=tokens, n=n, k=min(n, _log(rng, 1, 64)), dtype=dtype,
                    score=rng.choice(["softmax", "sigmoid"]), sequences=rng.choice([1, 1, min(tokens, _log(rng, 1, 64))]),
                    masked=rng.choice([0.0, 0.3]), filled=rng.random() < 0.5, base=rng.random() < 0.5, gradient=gradient,
                    add=gradient and rng.random() < 0.5, idx=idx)
    if kind in ("lookup", "embedding"):
        hd = rng.choice([64, 128, 512, 1024, 2048, rng.randint(1, 300), rng.randint(1, 2048)])
        case = dict(kind=kind, tokens=_log(rng, 1, min(65536, (1 << 26) // hd)), rows=_log(rng, 100, min(131072, (1 << 27) // hd)),
                    hd=hd, dtype=dtype, out=out, idx=idx)
        if kind == "embedding":
            case["accumulate"] = out == "f32" and rng.random() < 0.5
        return case
    hd, chunk = rng.choice([64, 128, 256, rng.randint(1, 300)]), rng.choice([1, 16, 64])
    width0, width1 = rng.randint(1, 96), rng.choice([0, rng.randint(1, 64)])
    most = max(1, min(65536, (1 << 28) // (hd * (width0 + width1))) // chunk)
    return dict(kind=kind, tokens=chunk * _log(rng, 1, most), n_slots=_log(rng, 1000, 1 << 19), hd=hd, width0=width0,
                width1=width1, chunk=chunk, ragged=chunk > 1, wdtype=dtype, out=out,
                accumulate=out == "f32" and rng.random() < 0.5, skewed=rng.random() < 0.5, idx=idx)


# ---------------------------------------------------------------- sizes

def _size(name):
    return {"bf16": 2, "f32": 4, "i32": 4, "i64": 8}[name]


def _touched(entries, rows, skewed):
    """How many of the rows `entries` draws of them meet, on average."""
    if not skewed:
        return rows * -math.expm1(entries * math.log1p(-1.0 / rows)) if rows > 1 else 1
    i = np.arange(1, rows + 1, dtype=np.float64)
    p = np.log1p(1 / i) / math.log(rows + 1)  # of number i among the tokens by frequency, as _skewed draws them
    return float(-np.expm1(entries * np.log1p(-np.minimum(p, 1 - 1e-12))).sum())


def _live(case):
    """Readings that are no padding."""
    return case["tokens"] * (case["chunk"] + 1) / (2 * case["chunk"]) if case["ragged"] else case["tokens"]


def work(case):
    kind, ib = case["kind"], _size(case["idx"])
    if kind == "balance":
        t, n, k, es = case["tokens"], case["n"], case["k"], _size(case["dtype"])
        entry = ib + (4 if case["filled"] else 0)
        passes = 1 + (1 + (1 if case["add"] else 0) if case["gradient"] else 0)
        return {"bytes": passes * t * n * es + t * k * entry + (ib * t if case["base"] else 0) + 4 * case["sequences"] * (n + 3),
                "flops": (10 if case["gradient"] else 6) * t * n}
    if kind in ("lookup", "embedding"):
        t, hd, es, os = case["tokens"], case["hd"], _size(case["dtype"]), _size(case["out"])
        rows = _touched(t, case["rows"], True)
        if kind == "lookup":
            return {"bytes": rows * hd * es + t * (ib + hd * os), "flops": t * hd}
        written = 2 * rows if case["accumulate"] else case["rows"]
        return {"bytes": t * (ib + hd * es) + written * hd * os, "flops": 2 * t * hd}
    live, width, hd = _live(case), case["width0"] + case["width1"], case["hd"]
    rows = _touched(live * width, case["n_slots"], case["skewed"])
    written = 2 * rows if case["accumulate"] else case["n_slots"]
    return {"bytes": live * (width * (ib + _size(case["wdtype"])) + (2 if case["width1"] else 1) * hd * 4) +
            written * hd * _size(case["out"]), "flops": 2 * live * width * hd}


# ---------------------------------------------------------------- inputs

def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _skewed(gen, rows, *shape):
    """Numbers below `rows` by a power law: the i-th most frequent about i times as rare as the first."""
    rank = torch.exp(torch.rand(shape, generator=gen, device="cuda", dtype=torch.float64) * math.log(rows + 1)).long() - 1
    return torch.randperm(rows, generator=gen, device="cuda")[rank.clamp_(0, rows - 1)]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case}
    kind, it = case["kind"], INDEX[case["idx"]]
    if kind == "balance":
        t, n, k, m = case["tokens"], case["n"], case["k"], case["sequences"]
        x = _normal(gen, t, n) * 2 + _normal(gen, n) * 0.5  # some entries are chosen more often than others
        if case["masked"]:
            x.masked_fill_(torch.rand((t, n), generator=gen, device="cuda") < case["masked"], -math.inf)
        s["logits"] = x.to(DTYPES[case["dtype"]])
        chosen = s["logits"].float().topk(k, dim=1)
        s["idx"], s["base"] = chosen.indices, None
        if case["base"]:
            s["base"] = (torch.arange(t, device="cuda") * n).to(it)
            s["idx"] = s["idx"] + s["base"].long()[:, None]
        s["idx"] = s["idx"].to(it)
        s["w"] = None
        if case["filled"]:  # weights of a router whose groups left fewer than k entries here and there
            w = torch.sigmoid(chosen.values)
            s["w"] = torch.where(torch.rand((t, k), generator=gen, device="cuda") < 0.1, torch.zeros_like(w), w)
        s["offsets"] = None
        if m > 1:  # sequences of different lengths, some empty; the last tokens belong to none
            cuts = torch.randint(0, t + 1, (m,), generator=gen, device="cuda").sort().values
            s["offsets"] = torch.cat([torch.zeros_like(cuts[:1]), cuts]).to(torch.int32)
        s["dloss"] = 0.01 * (1 + torch.rand(m, generator=gen, device="cuda"))
        s["add"] = (_normal(gen, t, n) / (t * n)).to(s["logits"].dtype) if case["add"] else None
    elif kind in ("lookup", "embedding"):
        t, rows, hd = case["tokens"], case["rows"], case["hd"]
        tokens = _skewed(gen, rows, t)
        s["padding"] = int(tokens[0]) if t > 8 else None  # a frequent one as a rule
        s["tokens"] = tokens.to(it)
        s["scale"] = math.sqrt(hd)
        if kind == "lookup":
            s["table"] = torch.cat([(_normal(gen, min(1 << 15, rows - r), hd) / math.sqrt(hd)).to(DTYPES[case["dtype"]])
                                    for r in range(0, rows, 1 << 15)])
        else:
            s["dout"] = (_normal(gen, t, hd) / t).to(DTYPES[case["dtype"]])
            s["grad"] = torch.zeros((rows, hd), device="cuda") if case["accumulate"] else None
    else:
        t, hd, n = case["tokens"], case["hd"], case["n_slots"]
        widths = [case["width0"]] + ([case["width1"]] if case["width1"] else [])
        s["valid"] = torch.randint(1, case["chunk"] + 1, (t // case["chunk"],), generator=gen, device="cuda",
                                   dtype=torch.int32) if case["ragged"] else None
        s["idx"] = [(_skewed(gen, n, t, w) if case["skewed"] else torch.randint(0, n, (t, w), generator=gen, device="cuda")).to(it)
                    for w in widths]
        s["w"] = [(_normal(gen, t, w) / 8).to(DTYPES[case["wdtype"]]) for w in widths]
        s["dout"] = [_normal(gen, t, hd) for _ in widths]
        s["grad"] = torch.zeros((n, hd), device="cuda") if case["accumulate"] else None
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    return (_own if own else _plain)[case["kind"]](state, case)


def _own_balance(s, c):
    from decode_state_gb300 import routing

    return routing.balance(s["logits"], s["idx"], score=c["score"], w=s["w"], base=s["base"], offsets=s["offsets"],
                           scale=1.5, gradient=c["gradient"], dloss=s["dloss"] if c["gradient"] else None, add=s["add"])


def _own_lookup(s, c):
    from decode_state_gb300 import embedding

    return embedding.lookup(s["table"], s["tokens"], scale=s["scale"], padding=s["padding"], dtype=DTYPES[c["out"]])


def _own_embedding(s, c):
    from decode_state_gb300 import embedding

    return embedding.backward(s["dout"], s["tokens"], c["rows"], scale=s["scale"], padding=s["padding"],
                              dtype=DTYPES[c["out"]], out=s["grad"], accumulate=c["accumulate"])


def _own_rows(s, c):
    from decode_state_gb300 import quant

    return quant.gather_drows(list(zip(s["idx"], s["w"], s["dout"])), c["n_slots"], chunk=c["chunk"], chunk_valid=s["valid"],
                              dtype=DTYPES[c["out"]], out=s["grad"], accumulate=c["accumulate"])


# ---------------------------------------------------------------- plain forms, in float32

def _sequence(s, c):
    """Each token's sequence, and the sequences' lengths; the tokens behind the last one get a number of their own."""
    if s["offsets"] is None:
        return torch.zeros(c["tokens"], dtype=torch.int64, device="cuda"), torch.full((1,), float(c["tokens"]), device="cuda")
    at = torch.arange(c["tokens"], device="cuda", dtype=torch.int32)
    return torch.searchsorted(s["offsets"], at, right=True) - 1, (s["offsets"][1:] - s["offsets"][:-1]).float()


def _plain_balance(s, c):
    n, m = c["n"], c["sequences"]
    seq, length = _sequence(s, c)
    x = s["logits"].float()
    masked = x.isnan() | (x == -math.inf)
    if c["score"] == "sigmoid":
        score = torch.where(masked, torch.zeros_like(x), 1 / (1 + torch.exp(-x)))
    else:
        x = torch.where(masked, torch.full_like(x, -math.inf), x)
        score = torch.where(masked, torch.zeros_like(x), torch.exp(x - x.amax(1, keepdim=True)))
    total = score.sum(1, keepdim=True)
    p = torch.where(total > 0, score / total, torch.zeros_like(score))
    idx = s["idx"].long()
    if s["base"] is not None:
        idx = idx - s["base"].long()[:, None]
    taken = torch.ones_like(idx, dtype=torch.int32) if s["w"] is None else (s["w"] != 0).to(torch.int32)
    counts = torch.zeros((m + 1) * n, dtype=torch.int32, device="cuda")
    counts.index_add_(0, (seq[:, None] * n + idx).view(-1), taken.view(-1))
    counts = counts.view(m + 1, n)[:m]
    share = torch.zeros((m + 1, n), device="cuda").index_add_(0, seq, p)[:m]
    both = length * counts.sum(1)
    factor = torch.where(both > 0, 1.5 * n / both, torch.zeros_like(both))
    loss = factor * (counts * share).sum(1)
    if not c["gradient"]:
        return loss, counts
    of = torch.cat([counts, torch.zeros_like(counts[:1])])[seq].float()
    g = torch.cat([factor * s["dloss"], torch.zeros_like(factor[:1])])[seq][:, None]
    d = g * p * (of - (p * of).sum(1, keepdim=True))
    if c["score"] == "sigmoid":
        d = d * (1 - score)
    if s["add"] is not None:
        d = d + s["add"].float()
    return loss, counts, d.to(s["logits"].dtype)


def _plain_lookup(s, c):
    tokens = s["tokens"].long()
    out = s["table"][tokens].float() * s["scale"]
    if s["padding"] is not None:
        out = torch.where((tokens == s["padding"])[:, None], torch.zeros_like(out), out)
    return out.to(DTYPES[c["out"]])


def _plain_embedding(s, c):
    tokens = s["tokens"].long()
    d = s["dout"].float() * s["scale"]
    if s["padding"] is not None:
        d = torch.where((tokens == s["padding"])[:, None], torch.zeros_like(d), d)
    if c["accumulate"]:
        return s["grad"].index_add_(0, tokens, d)
    return torch.zeros((c["rows"], c["hd"]), device="cuda").index_add_(0, tokens, d).to(DTYPES[c["out"]])


def _padding(s, c):
    """[tokens, 1]: which readings are no padding."""
    if s["valid"] is None:
        return torch.ones((c["tokens"], 1), dtype=torch.bool, device="cuda")
    at = torch.arange(c["tokens"], device="cuda")
    return (at % c["chunk"] < s["valid"][at // c["chunk"]])[:, None]


def _plain_rows(s, c):
    grad = s["grad"] if c["accumulate"] else torch.zeros((c["n_slots"], c["hd"]), device="cuda")
    live = _padding(s, c)
    for idx, w, dout in zip(s["idx"], s["w"], s["dout"]):
        w = torch.where(live, w.float(), torch.zeros((), device="cuda"))
        grad.index_add_(0, idx.long().view(-1), (w[..., None] * dout[:, None]).view(-1, c["hd"]))
    return grad if c["accumulate"] else grad.to(DTYPES[c["out"]])


_plain = {"balance": _plain_balance, "lookup": _plain_lookup, "embedding": _plain_embedding, "rows": _plain_rows}
_own = {"balance": _own_balance, "lookup": _own_lookup, "embedding": _own_embedding, "rows": _own_rows}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_balance(s, c):
    n, k = c["n"], c["k"]
    ends = [0, c["tokens"]] if s["offsets"] is None else s["offsets"].tolist()
    idx = s["idx"].long()
    if s["base"] is not None:
        idx = idx - s["base"].long().unsqueeze(1)
    weight = torch.ones(idx.shape, dtype=torch.float64, device="cuda") if s["w"] is None else (s["w"] != 0).double()
    losses, grad = [], torch.zeros(s["logits"].shape, dtype=torch.float64, device="cuda")
    for q, (a, b) in enumerate(zip(ends[:-1], ends[1:])):
        if a == b:
            losses.append(torch.zeros((), dtype=torch.float64, device="cuda"))
            continue
        with torch.enable_grad():  # the derivative that automatic differentiation finds
            x = s["logits"][a:b].double().requires_grad_()
            dead = x.detach() == -math.inf
            live = torch.where(dead, torch.full_like(x, -1e4), x)
            score = torch.sigmoid(live) if c["score"] == "sigmoid" else torch.softmax(live, 1)
            score = torch.where(dead, torch.zeros_like(score), score)
            share = (score / score.sum(1, keepdim=True).clamp_min(1e-300)).mean(0)
            count = torch.bincount(idx[a:b].reshape(-1), weights=weight[a:b].reshape(-1), minlength=n)
            loss = 1.5 * n * (count / count.sum().clamp_min(1) * share).sum()
        if c["gradient"]:
            loss.backward(s["dloss"][q].double())
            grad[a:b] = x.grad
        losses.append(loss.detach())
    losses = torch.stack(losses)
    if not c["gradient"]:
        return losses, None
    return losses, None, grad if s["add"] is None else grad + s["add"].double()


def _exact_lookup(s, c):
    keep = torch.ones(c["rows"], dtype=torch.float64, device="cuda")
    if s["padding"] is not None:
        keep[s["padding"]] = 0
    tokens = s["tokens"].long()
    return torch.cat([s["table"].index_select(0, t).double() * (keep[t] * s["scale"]).unsqueeze(1) for t in tokens.split(1 << 14)])


def _by_row(rows, at, values):
    """Add the values [m, hd] to their rows: sorted by row, then a sum over each run of equal ones."""
    at, order = at.sort()
    unique, length = at.unique_consecutive(return_counts=True)
    rows[unique] += torch.segment_reduce(values[order], "sum", lengths=length, axis=0, unsafe=True)


def _exact_embedding(s, c):
    grad = torch.zeros((c["rows"], c["hd"]), dtype=torch.float64, device="cuda")
    at = s["tokens"].long()
    keep = torch.arange(len(at), device="cuda") if s["padding"] is None else (at != s["padding"]).nonzero().squeeze(1)
    if len(keep):
        _by_row(grad, at[keep], s["dout"][keep].double() * s["scale"])
    return grad


def _exact_rows(s, c):
    grad = torch.zeros((c["n_slots"], c["hd"]), dtype=torch.float64, device="cuda")
    at = torch.arange(c["tokens"], device="cuda")
    live = at if s["valid"] is None else at[at % c["chunk"] < s["valid"].long().repeat_interleave(c["chunk"])]
    for idx, w, dout in zip(s["idx"], s["w"], s["dout"]):
        for t in live.split(max(1, (1 << 27) // (idx.shape[1] * c["hd"]))):
            values = w[t].double().unsqueeze(2) * dout[t].double().unsqueeze(1)
            _by_row(grad, idx[t].long().flatten(), values.flatten(0, 1))
    return grad


def exact(case, seed):
    return {"balance": _exact_balance, "lookup": _exact_lookup, "embedding": _exact_embedding,
            "rows": _exact_rows}[case["kind"]](prepare(case, seed), case)
