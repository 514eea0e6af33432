"""The routing and quantised-cache operators: what is measured, on which inputs, and their plain forms.

Four operators, in the order in which a layer runs them:
  route   scores -> slots and weights (softmax or sigmoid, balance bias, groups, top-k), and its gradient
  cache   rows quantised as they are written into the bank's slots, and read back
  gather  weighted sums of quantised bank rows, and the gradient of the weights
  decode  write-then-read tokens on a quantised bank

``own`` chooses between the framework's kernels and plain forms in elementary float32 operations.
"""

from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
INDEX = {"i32": torch.int32, "i64": torch.int64}
LEVELS = {"int8": 127.0, "fp8": 448.0, "int4": 7.0}  # the largest code of each format
TINY = 2.0 ** -100  # a group whose largest magnitude is below this is stored as zeros


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the router of one decoding step: 64 streams, 256 entries in 8 groups, 8 of them chosen; latency counts
        dict(name="route step", kind="route", tokens=64, n=256, k=8, dtype="bf16", score="sigmoid", bias=True,
             groups=8, top_groups=4, group_top=2, renorm=True, scale=1.5, masked=0.0, base=False, idx="i32"),
        # the same router over a prompt or a training batch
        dict(name="route prompt", kind="route", tokens=65536, n=256, k=8, dtype="bf16", score="sigmoid", bias=True,
             groups=8, top_groups=4, group_top=2, renorm=True, scale=1.5, masked=0.0, base=False, idx="i32"),
        # the serving decode's addressing: 1024 streams choose 64 of their own 16384 slots, a quarter not in use yet
        dict(name="route slots", kind="route", tokens=1024, n=16384, k=64, dtype="f32", score="softmax", bias=False,
             groups=1, top_groups=1, group_top=1, renorm=True, scale=1.0, masked=0.25, base=True, idx="i32"),
        # training a router of ragged size whose weights are not renormalised: every logit has a gradient
        dict(name="route gradient", kind="route_grad", tokens=4097, n=4099, k=33, dtype="f32", score="softmax",
             renorm=False, scale=1.0, masked=0.02, idx="i64"),
        # the rows that one step of 64 streams writes, ragged columns
        dict(name="cache step", kind="cache", rows=2048, n_slots=65536, hd=136, group=64, format="int8", dtype="bf16",
             idx="i64"),
        # a prompt's bank turned into a 4-bit snapshot
        dict(name="cache prompt", kind="cache", rows=1 << 20, n_slots=1 << 21, hd=128, group=32, format="int4",
             dtype="f32", idx="i32"),
        # one slab of 256 tokens out of a large bank
        dict(name="gather slab", kind="gather", tokens=256, n_slots=1 << 22, hd=128, group=128, format="int8",
             width0=64, width1=0, chunk=1, ragged=False, wdtype="bf16", idx="i64"),
        # the framework's gather workload on an 8-bit bank: two operands, chunks with padding
        dict(name="gather batch", kind="gather", tokens=65536, n_slots=1 << 22, hd=128, group=128, format="fp8",
             width0=64, width1=64, chunk=64, ragged=True, wdtype="bf16", idx="i64"),
        # the weights' gradient over an unquantised bank of odd sizes
        dict(name="gradient ragged", kind="gather_dw", tokens=1000, n_slots=100003, hd=264, group=128, format="bf16",
             width0=37, width1=0, chunk=1, ragged=False, wdtype="f32", idx="i32"),
        # the weights' gradient of the gather workload
        dict(name="gradient batch", kind="gather_dw", tokens=65536, n_slots=1 << 22, hd=128, group=128, format="int8",
             width0=64, width1=0, chunk=64, ragged=True, wdtype="bf16", idx="i64"),
        # one token of 64 streams with a gate for each write; the rows written are read back
        dict(name="decode step", kind="decode", streams=64, slots=4096, hd=128, group=128, format="int8", W=32, R=32,
             per_write=True, T=1, whole=False, idx="i64"),
        # 32 tokens of 512 streams in one call, then the state as bf16
        dict(name="decode tokens", kind="decode", streams=512, slots=1024, hd=128, group=64, format="fp8", W=64, R=64,
             per_write=False, T=32, whole=True, idx="i32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["route", "route", "route_grad", "cache", "gather", "gather_dw", "decode"])
    idx = rng.choice(["i32", "i64"])
    dtype = rng.choice(["bf16", "f32"])
    if kind in ("route", "route_grad"):
        groups = rng.choice([1, 1, 2, 4, 8]) if kind == "route" else 1
        n = groups * _log(rng, 8, 16384 // groups)
        least = 1 if kind == "route" else 8  # one chosen entry, renormalised, has no gradient: nothing to compare
        tokens = _log(rng, least, min(65536, (1 << 24) // n))
        score = rng.choice(["softmax", "sigmoid"])
        case = dict(kind=kind, tokens=tokens, n=n, k=min(n, _log(rng, min(2, least), 64)), dtype=dtype, score=score,
                    renorm=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]), masked=rng.choice([0.0, 0.3]), idx=idx)
        if kind == "route":
            case.update(bias=score == "sigmoid" and rng.random() < 0.5, groups=groups,
                        top_groups=rng.randint(1, groups), group_top=rng.choice([1, 2]), base=rng.random() < 0.5)
        return case
    hd = rng.choice([64, 128, 256, rng.randint(1, 300)])
    group = rng.choice([32, 64, 128])
    if kind == "cache":
        rows = _log(rng, 1, (1 << 19) if hd <= 128 else (1 << 18))
        return dict(kind=kind, rows=rows, n_slots=rows + rng.randint(0, rows), hd=hd, group=group,
                    format=rng.choice(["int8", "fp8", "int4"]), dtype=dtype, idx=idx)
    if kind in ("gather", "gather_dw"):
        chunk = rng.choice([1, 16, 64])
        most = max(1, min(65536, (1 << 23) // hd) // chunk)
        formats = ["int8", "fp8", "int4"] + (["bf16", "f32"] if kind == "gather_dw" else [])
        return dict(kind=kind, tokens=chunk * _log(rng, 1, most), n_slots=_log(rng, 1000, 1 << 19), hd=hd, group=group,
                    format=rng.choice(formats), width0=rng.randint(1, 96), width1=rng.choice([0, rng.randint(1, 64)]),
                    chunk=chunk, ragged=chunk > 1, wdtype=dtype, idx=idx)
    W, R, T = rng.randint(1, 96), rng.randint(1, 96), rng.choice([1, 1, rng.randint(2, 16)])
    slots = _log(rng, 100, 1024)
    return dict(kind=kind, streams=_log(rng, 1, 512), slots=slots, hd=hd, group=group,
                format=rng.choice(["int8", "fp8"]), W=W, R=R, per_write=rng.random() < 0.5, T=T, whole=T > 1, idx=idx)


# ---------------------------------------------------------------- sizes

def _payload(hd, fmt):
    return {"int4": (hd + 1) // 2, "bf16": 2 * hd, "f32": 4 * hd}.get(fmt, hd)


def _pitch(hd, fmt):
    """Bytes from one quantised row to the next: the codes, padded to 16 bytes."""
    return (_payload(hd, fmt) + 15) // 16 * 16


def _row_bytes(case):
    """A bank row as it is read or written: its codes and scales."""
    fmt = case["format"]
    return _payload(case["hd"], fmt) + (4 * -(-case["hd"] // case["group"]) if fmt in LEVELS else 0)


def work(case):
    kind, ib = case["kind"], 4 if case["idx"] == "i32" else 8
    if kind == "route":
        es = 2 if case["dtype"] == "bf16" else 4
        t, n, k = case["tokens"], case["n"], case["k"]
        return {"bytes": t * n * es + t * k * (ib + 4) + (4 * n if case["bias"] else 0) + (ib * t if case["base"] else 0),
                "flops": 4 * t * n}
    if kind == "route_grad":
        es = 2 if case["dtype"] == "bf16" else 4
        t, n, k = case["tokens"], case["n"], case["k"]
        read = n if case["score"] == "softmax" and not case["renorm"] else k
        return {"bytes": t * (n + read) * es + t * k * (ib + 4), "flops": 4 * t * read}
    if kind == "cache":
        es = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": case["rows"] * (case["hd"] * (es + 2) + _row_bytes(case) + ib), "flops": 4 * case["rows"] * case["hd"]}
    if kind in ("gather", "gather_dw"):
        widths = [case["width0"]] + ([case["width1"]] if case["width1"] else [])
        live = case["tokens"] * (case["chunk"] + 1) / (2 * case["chunk"]) if case["ragged"] else case["tokens"]
        wb = 2 if case["wdtype"] == "bf16" else 4
        entries = live * sum(widths)
        rows = min(entries, case["n_slots"]) * _row_bytes(case)
        side = case["tokens"] * len(widths) * case["hd"] * 4 * (1 if kind == "gather" else live / case["tokens"])
        dw = case["tokens"] * sum(widths) * wb if kind == "gather_dw" else entries * wb
        return {"bytes": rows + entries * ib + dw + side, "flops": 2 * entries * case["hd"]}
    S, T, W, R, hd = case["streams"], case["T"], case["W"], case["R"], case["hd"]
    held = S * case["slots"]
    rows = (min(S * T * (W + R), held) + min(S * T * W, held)) * _row_bytes(case)
    inputs = S * T * ((W + R) * (ib + 4) + hd * 4 + 4 + 4 * (W if case["per_write"] else 1) + hd * 2)
    back = (held if case["whole"] else S * W) * hd * 2
    return {"bytes": rows + inputs + back, "flops": S * T * hd * (6 * W + 2 * R)}


# ---------------------------------------------------------------- inputs

def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _bank(gen, n_slots, hd, group, fmt, std=1.0):
    """A bank of normal rows: (codes, scales), or (rows, None) for an unquantised one."""
    if fmt in DTYPES:
        return torch.cat([(_normal(gen, min(1 << 20, n_slots - r), hd) * std).to(DTYPES[fmt])
                          for r in range(0, n_slots, 1 << 20)]), None
    parts = [_quantise(_normal(gen, min(1 << 20, n_slots - r), hd) * std, group, fmt) for r in range(0, n_slots, 1 << 20)]
    return torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])


def _distinct(gen, rows, k, n):
    """[rows, k] numbers below n, distinct within a row: increasing ones with random gaps, shuffled."""
    gaps = torch.rand((rows, k), generator=gen, device="cuda").cumsum(1)
    scaled = gaps / (gaps[:, -1:] + torch.rand((rows, 1), generator=gen, device="cuda")) * (n - k)
    ordered = scaled.to(torch.int64).clamp_(0, n - k) + torch.arange(k, device="cuda")
    return ordered.gather(1, torch.rand((rows, k), generator=gen, device="cuda").argsort(1))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case}
    kind, it = case["kind"], INDEX[case["idx"]]
    if kind in ("route", "route_grad"):
        t, n, k = case["tokens"], case["n"], case["k"]
        x = _normal(gen, t, n) * 2
        if case["masked"]:
            x.masked_fill_(torch.rand((t, n), generator=gen, device="cuda") < case["masked"], -math.inf)
        s["logits"] = x.to(DTYPES[case["dtype"]])
        if kind == "route":
            s["bias"] = _normal(gen, n) * 0.1 if case["bias"] else None
            s["base"] = (torch.arange(t, device="cuda") * n).to(it) if case["base"] else None
        else:
            s["idx"] = s["logits"].float().topk(k, dim=1).indices.to(it)
            s["dw"] = _normal(gen, t, k)
    elif kind == "cache":
        s["rows"] = (_normal(gen, case["rows"], case["hd"]) * torch.exp(_normal(gen, case["rows"], 1))).to(DTYPES[case["dtype"]])
        s["slots"] = torch.randperm(case["n_slots"], generator=gen, device="cuda")[:case["rows"]].to(it)
        s["codes"] = torch.zeros((case["n_slots"], _pitch(case["hd"], case["format"])), dtype=torch.uint8, device="cuda")
        s["scales"] = torch.zeros((case["n_slots"], -(-case["hd"] // case["group"])), device="cuda")
    elif kind in ("gather", "gather_dw"):
        t, hd = case["tokens"], case["hd"]
        s["codes"], s["scales"] = _bank(gen, case["n_slots"], hd, case["group"], case["format"])
        widths = [case["width0"]] + ([case["width1"]] if case["width1"] else [])
        s["valid"] = torch.randint(1, case["chunk"] + 1, (t // case["chunk"],), generator=gen, device="cuda",
                                   dtype=torch.int32) if case["ragged"] else None
        s["idx"] = [torch.randint(0, case["n_slots"], (t, w), generator=gen, device="cuda").to(it) for w in widths]
        if kind == "gather":
            s["w"] = [(_normal(gen, t, w) / 8).to(DTYPES[case["wdtype"]]) for w in widths]
        else:
            s["dout"] = [_normal(gen, t, hd) for _ in widths]
    else:
        S, T, W, R, hd, P = case["streams"], case["T"], case["W"], case["R"], case["hd"], case["slots"]
        s["codes"], s["scales"] = _bank(gen, S * P, hd, case["group"], case["format"], 0.3)
        base = (torch.arange(S, device="cuda") * P).view(1, S, 1)
        s["k_idx"] = (_distinct(gen, T * S, W, P).view(T, S, W) + base).to(it)
        s["k_val"] = torch.nn.functional.normalize(_normal(gen, T, S, W), dim=-1)  # unit keys, as the layer makes them
        s["v"] = _normal(gen, T, S, hd)
        s["beta"] = torch.sigmoid(_normal(gen, T, S))
        s["g"] = -torch.nn.functional.softplus(_normal(gen, T, S, W if case["per_write"] else 1) - 2)
        s["q_idx"] = (torch.randint(0, P, (T, S, R), generator=gen, device="cuda") + base).to(it)
        s["q_val"] = torch.nn.functional.normalize(_normal(gen, T, S, R), dim=-1)
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    return (_own if own else _plain)[case["kind"]](state, case)


def _own_route(s, c):
    from decode_state_gb300 import routing

    return routing.route(s["logits"], c["k"], score=c["score"], bias=s["bias"], groups=c["groups"],
                         top_groups=c["top_groups"], group_top=c["group_top"], renorm=c["renorm"], scale=c["scale"],
                         base=s["base"], idx_dtype=INDEX[c["idx"]])


def _own_route_grad(s, c):
    from decode_state_gb300 import routing

    return routing.route_backward(s["logits"], s["idx"], s["dw"], score=c["score"], renorm=c["renorm"], scale=c["scale"])


def _handle(s, c):
    from decode_state_gb300 import quant

    if c["format"] in DTYPES:
        return s["codes"]
    return quant.QuantBank(s["codes"], s["scales"], c["hd"], group=c["group"], format=c["format"])


def _own_cache(s, c):
    from decode_state_gb300 import quant

    bank = _handle(s, c)
    quant.quantize_rows(bank, s["rows"], s["slots"])
    return quant.dequantize_rows(bank, s["slots"], dtype=torch.bfloat16)


def _own_gather(s, c):
    from decode_state_gb300 import quant

    return quant.gather(_handle(s, c), list(zip(s["idx"], s["w"])), chunk=c["chunk"], chunk_valid=s["valid"])


def _own_gather_dw(s, c):
    from decode_state_gb300 import quant

    return quant.gather_dw(_handle(s, c), list(zip(s["idx"], s["dout"])), chunk=c["chunk"], chunk_valid=s["valid"],
                           dtype=DTYPES[c["wdtype"]])


def _own_decode(s, c):
    from decode_state_gb300 import quant

    bank = _handle(s, c)
    args = [s[n] for n in ("k_idx", "k_val", "v", "beta", "g", "q_idx", "q_val")]
    if c["T"] == 1:
        out = quant.decode_step(bank, *(a[0] for a in args), out_dtype=torch.bfloat16)[None]
    else:
        out = quant.decode_seq(bank, *args, out_dtype=torch.bfloat16)
    return out, quant.dequantize_rows(bank, None if c["whole"] else s["k_idx"].view(-1), dtype=torch.bfloat16)


# ---------------------------------------------------------------- plain forms, in float32

def _quantise(x, group, fmt):
    """Rows [m, hd] -> (codes [m, pitch] as bytes, scales [m, groups])."""
    m, hd = x.shape
    groups = -(-hd // group)
    x = torch.nn.functional.pad(x, (0, groups * group - hd)).view(m, groups, group)
    amax = x.abs().amax(2, keepdim=True)
    amax = torch.where(amax < TINY, torch.zeros_like(amax), amax)
    top = torch.full_like(amax, LEVELS[fmt])
    y = torch.where(amax > 0, x * (top / amax), torch.zeros_like(x))
    scales = (amax / top).view(m, groups)
    y = y.view(m, groups * group)[:, :hd]
    if fmt == "fp8":
        codes = y.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        codes = y.round().clamp_(-LEVELS[fmt], LEVELS[fmt]).to(torch.int8).view(torch.uint8)
    if fmt == "int4":
        codes = torch.nn.functional.pad(codes, (0, hd % 2))
        codes = (codes[:, 0::2] & 15) | (codes[:, 1::2] << 4)
    return torch.nn.functional.pad(codes, (0, _pitch(hd, fmt) - codes.shape[1])), scales


def _values(codes, scales, hd, group, fmt):
    """The float32 rows that codes [..., pitch] and scales [..., groups] stand for."""
    if fmt in DTYPES:
        return codes.float()
    if fmt == "int4":
        nibbles = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).to(torch.int32)
        y = ((nibbles ^ 8) - 8).float()[..., :hd]
    elif fmt == "fp8":
        y = codes[..., :hd].view(torch.float8_e4m3fn).float()
    else:
        y = codes[..., :hd].view(torch.int8).float()
    return y * scales.repeat_interleave(group, -1)[..., :hd]


def _bank_rows(s, c, idx):
    idx = idx.long()
    scales = s["scales"][idx] if s["scales"] is not None else None
    return _values(s["codes"][idx], scales, c["hd"], c["group"], c["format"])


def _scores(x, score):
    """(scores, exp(x - max) for a softmax, the masked entries)."""
    masked = x.isnan() | (x == -math.inf)
    if score == "sigmoid":
        s = 1 / (1 + torch.exp(-x))
        return torch.where(masked, torch.zeros_like(s), s), None, masked
    x = torch.where(masked, torch.full_like(x, -math.inf), x)
    top = x.amax(1, keepdim=True)
    e = torch.where(masked, torch.zeros_like(x), torch.exp(x - top))
    total = e.sum(1, keepdim=True)
    return torch.where(total > 0, e / total, torch.zeros_like(e)), e, masked


def _plain_route(s, c):
    x = s["logits"].float()
    score, e, masked = _scores(x, c["score"])
    if s["bias"] is not None:
        key = score + s["bias"]
    else:
        key = x if c["score"] == "softmax" else score
    none = torch.full_like(key, -math.inf)
    key = torch.where(masked, none, key)
    if c["groups"] > 1 and c["top_groups"] < c["groups"]:
        by_group = key.view(len(key), c["groups"], -1)
        if c["group_top"] == 1:
            rank = by_group.amax(2)
        else:
            raw = key if s["bias"] is not None or e is None else torch.where(masked, none, e)
            best = raw.view(by_group.shape).sort(dim=2, descending=True).values[..., :2]
            rank = torch.where(best == -math.inf, torch.zeros_like(best), best).sum(2)
            rank = torch.where(best[..., 0] == -math.inf, torch.full_like(rank, -math.inf), rank)
        order = rank.sort(dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        kept = torch.zeros_like(rank, dtype=torch.bool).scatter_(1, order, True)
        key = torch.where(kept[..., None], by_group, none.view(by_group.shape)).view(key.shape)
    ranked = key.sort(dim=1, descending=True, stable=True)
    idx = ranked.indices[:, :c["k"]]
    w = torch.where(ranked.values[:, :c["k"]] == -math.inf, torch.zeros((), device=x.device), score.gather(1, idx))
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
    if s["base"] is not None:
        idx = idx + s["base"].long()[:, None]
    return idx.to(INDEX[c["idx"]]), w * c["scale"]


def _plain_route_grad(s, c):
    x = s["logits"].float()
    score, _, _ = _scores(x, c["score"])
    idx, dw = s["idx"].long(), s["dw"] * c["scale"]
    chosen = score.gather(1, idx)
    if c["renorm"]:
        total = chosen.sum(1, keepdim=True)
        w = torch.where(total > 0, chosen / total, torch.zeros_like(chosen))
        dw = torch.where(total > 0, (dw - (dw * w).sum(1, keepdim=True)) / total, torch.zeros_like(dw))
    if c["score"] == "sigmoid":
        dx = torch.zeros_like(x).scatter_(1, idx, dw * chosen * (1 - chosen))
    else:
        mean = (dw * chosen).sum(1, keepdim=True)
        if c["renorm"]:
            mean = torch.zeros_like(mean)  # the sum over the chosen of dw * s vanishes
        dx = score * (torch.zeros_like(x).scatter_(1, idx, dw) - mean)
    return dx.to(s["logits"].dtype)


def _plain_cache(s, c):
    slots = s["slots"].long()
    s["codes"][slots], s["scales"][slots] = _quantise(s["rows"].float(), c["group"], c["format"])
    return _bank_rows(s, c, slots).to(torch.bfloat16)


def _live(s, c):
    """[tokens, 1]: which tokens are no padding."""
    if s["valid"] is None:
        return torch.ones((c["tokens"], 1), dtype=torch.bool, device="cuda")
    at = torch.arange(c["tokens"], device="cuda")
    return (at % c["chunk"] < s["valid"][at // c["chunk"]])[:, None]


def _plain_gather(s, c):
    live = _live(s, c)
    return [torch.where(live, (w.float()[..., None] * _bank_rows(s, c, idx)).sum(1), torch.zeros((), device="cuda"))
            for idx, w in zip(s["idx"], s["w"])]


def _plain_gather_dw(s, c):
    live = _live(s, c)
    return [torch.where(live, (dout[:, None] * _bank_rows(s, c, idx)).sum(2), torch.zeros((), device="cuda")).to(DTYPES[c["wdtype"]])
            for idx, dout in zip(s["idx"], s["dout"])]


def _plain_decode(s, c):
    out = []
    for t in range(c["T"]):  # every token reads what the one before it wrote
        k_idx = s["k_idx"][t].long()
        decayed = _bank_rows(s, c, k_idx) * torch.exp(s["g"][t])[..., None]
        k = s["k_val"][t][..., None]
        delta = s["beta"][t][:, None] * (s["v"][t] - (k * decayed).sum(1))
        new = decayed + k * delta[:, None]
        flat = k_idx.view(-1)
        s["codes"][flat], s["scales"][flat] = _quantise(new.view(-1, c["hd"]), c["group"], c["format"])
        out.append((s["q_val"][t][..., None] * _bank_rows(s, c, s["q_idx"][t])).sum(1).to(torch.bfloat16))
    rows = torch.arange(len(s["codes"]), device="cuda") if c["whole"] else s["k_idx"].view(-1)
    return torch.stack(out), _bank_rows(s, c, rows).to(torch.bfloat16)


_plain = {"route": _plain_route, "route_grad": _plain_route_grad, "cache": _plain_cache, "gather": _plain_gather,
          "gather_dw": _plain_gather_dw, "decode": _plain_decode}
_own = {"route": _own_route, "route_grad": _own_route_grad, "cache": _own_cache, "gather": _own_gather,
        "gather_dw": _own_gather_dw, "decode": _own_decode}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_rows(c, codes, scales):
    """Float64 rows of a bank's codes, by their definition: a table of the 256 bytes' values."""
    if c["format"] in DTYPES:
        return codes.double()
    b = torch.arange(256, device="cuda")
    if c["format"] == "fp8":
        e, m = (b >> 3) & 15, (b & 7).double()
        mag = torch.where(e > 0, (1 + m / 8) * torch.exp2((e - 7).double()), m / 8 * 2.0 ** -6)
        table = torch.where(b >= 128, -mag, mag)[:, None]
    elif c["format"] == "int8":
        table = torch.where(b >= 128, b - 256, b).double()[:, None]
    else:
        signed = lambda v: torch.where(v >= 8, v - 16, v).double()  # noqa: E731
        table = torch.stack([signed(b % 16), signed(b // 16)], 1)
    y = table[codes.long()].flatten(-2)[..., :c["hd"]]
    col = torch.arange(c["hd"], device="cuda") // c["group"]
    return y * scales.double()[..., col]


def _exact_round(c, x):
    """Float64 rows [m, hd] -> the values that they are held as."""
    col = torch.arange(c["hd"], device="cuda") // c["group"]
    top = torch.zeros((len(x), -(-c["hd"] // c["group"])), dtype=torch.float64, device="cuda")
    top = top.scatter_reduce_(1, col.expand_as(x), x.abs(), "amax")[:, col]
    top = torch.where(top < TINY, torch.zeros_like(top), top)
    scale = top / LEVELS[c["format"]]
    y = torch.where(top > 0, x / scale, torch.zeros_like(x))
    if c["format"] == "fp8":  # 3 bits behind the leading one, in steps of 2^-9 below 2^-6
        step = torch.exp2((torch.frexp(y.abs().clamp_min(2.0 ** -6)).exponent - 4).double())
        return torch.round(y / step) * step * scale
    return torch.round(y) * scale


def _exact_scores(x, score):
    x = torch.where(x.isnan(), torch.full_like(x, -math.inf), x)
    if score == "sigmoid":
        return torch.sigmoid(x)
    return torch.softmax(x, 1).nan_to_num(0.0)  # a row that is masked throughout


def _exact_route(s, c):
    x = s["logits"].double()
    score = _exact_scores(x, c["score"])
    key = score + s["bias"].double() if s["bias"] is not None else score
    key = torch.where(x == -math.inf, torch.full_like(key, -2.0), key)  # keys are above -1: biases are small
    if c["groups"] > 1:
        per = c["n"] // c["groups"]
        best = key.reshape(-1, c["groups"], per).topk(min(c["group_top"], per), 2).values
        rank = torch.where(best[..., 0] == -2.0, torch.full_like(best[..., 0], -9.0), best.clamp_min(-1.0).sum(2) + (best == -2.0).sum(2))
        drop = rank.sort(dim=1, descending=True, stable=True).indices[:, c["top_groups"]:]
        key = key.reshape(-1, c["groups"], per).scatter(1, drop[..., None].expand(-1, -1, per), -2.0).flatten(1)
    key, idx = key.sort(dim=1, descending=True, stable=True)
    w = score.gather(1, idx[:, :c["k"]]).masked_fill(key[:, :c["k"]] == -2.0, 0.0)
    if c["renorm"]:
        w = (w / w.sum(1, keepdim=True)).nan_to_num(0.0)
    return [None, w * c["scale"]]


def _exact_route_grad(s, c):
    with torch.enable_grad():  # the derivative that automatic differentiation finds
        x = s["logits"].double().requires_grad_()
        live = torch.where(x.detach() == -math.inf, torch.full_like(x, -1e4), x)
        score = torch.sigmoid(live) if c["score"] == "sigmoid" else torch.softmax(live, 1)
        w = score.gather(1, s["idx"].long())
        if c["renorm"]:
            w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
        (w * c["scale"] * s["dw"].double()).sum().backward()
    return x.grad.nan_to_num(0.0)


def _exact_cache(s, c):
    parts = s["rows"].split(1 << 18)
    return torch.cat([_exact_round(c, p.double()) for p in parts])


def _exact_gather(s, c):
    live, out = _live(s, c), []
    for idx, w in zip(s["idx"], s["w"]):
        out.append(torch.cat([(w[t:t + 4096].double().unsqueeze(1) @ _exact_rows(c, *_at(s, idx[t:t + 4096]))).squeeze(1)
                              for t in range(0, c["tokens"], 4096)]) * live)
    return out


def _exact_gather_dw(s, c):
    live, out = _live(s, c), []
    for idx, d in zip(s["idx"], s["dout"]):
        out.append(torch.cat([(_exact_rows(c, *_at(s, idx[t:t + 4096])) @ d[t:t + 4096].double().unsqueeze(2)).squeeze(2)
                              for t in range(0, c["tokens"], 4096)]) * live)
    return out


def _at(s, idx):
    idx = idx.long()
    return s["codes"][idx], s["scales"][idx] if s["scales"] is not None else None


def _exact_decode(s, c):
    bank = torch.cat([_exact_rows(c, a, b) for a, b in zip(s["codes"].split(1 << 18), s["scales"].split(1 << 18))])
    out = []
    for t in range(c["T"]):
        k_idx, k = s["k_idx"][t].long(), s["k_val"][t].double()
        rows = bank[k_idx] * s["g"][t].double().exp().unsqueeze(2)
        delta = s["beta"][t].double().unsqueeze(1) * (s["v"][t].double() - (k.unsqueeze(1) @ rows).squeeze(1))
        rows = rows + k.unsqueeze(2) * delta.unsqueeze(1)
        bank[k_idx.view(-1)] = _exact_round(c, rows.flatten(0, 1))
        out.append((s["q_val"][t].double().unsqueeze(1) @ bank[s["q_idx"][t].long()]).squeeze(1))
    return torch.stack(out), bank if c["whole"] else bank[s["k_idx"].long().view(-1)]


def exact(case, seed):
    if case["kind"] == "gather" or case["kind"] == "gather_dw":
        if case["tokens"] * (case["width0"] + case["width1"]) * case["hd"] > 1 << 31:
            return None
    return {"route": _exact_route, "route_grad": _exact_route_grad, "cache": _exact_cache, "gather": _exact_gather,
            "gather_dw": _exact_gather_dw, "decode": _exact_decode}[case["kind"]](prepare(case, seed), case)
