"""Plain float64 forms, on the CPU, of the balance loss, the embedding lookup and the gradients of rows."""

from __future__ import annotations

import torch

STEP = 2.0 ** -24  # one float32 rounding, relative


def half_step(dtype) -> float:
    """The largest relative error of one rounding to a type."""
    return torch.finfo(dtype).eps / 2


def shares(logits: torch.Tensor, score: str):
    """(p, 1 - s or 1 for a softmax) [tokens, n]: a row's scores over their sum; masked entries, and rows of nothing else,
    have 0, and several +inf share a softmax evenly."""
    x = logits.double()
    masked = x.isnan() | (x == -torch.inf)
    if score == "sigmoid":
        # scores over their sum, both scaled so that neither is lost: log s = min(x, 0) - log(1 + e^-|x|)
        log = torch.where(x > 0, torch.zeros_like(x), x) - torch.log1p(torch.exp(-x.abs()))
        rest = 1 / (1 + torch.exp(x))
    else:
        log, rest = x, torch.ones_like(x)
    log = torch.where(masked, torch.full_like(x, -torch.inf), log)
    top = log.amax(1, keepdim=True)
    s = torch.where(masked, torch.zeros_like(x), torch.where(log == top, torch.ones_like(x), torch.exp(log - top)))
    total = s.sum(1, keepdim=True)
    return torch.where(total > 0, s / total.clamp_min(1e-300), torch.zeros_like(s)), torch.where(masked, torch.zeros_like(x), rest)


def sequences(tokens: int, offsets):
    ends = [0, tokens] if offsets is None else [int(o) for o in offsets]
    return list(zip(ends[:-1], ends[1:]))


def count(idx, n, *, w=None, base=None, offsets=None):
    """counts [sequences, n] int64."""
    j = idx.long() - (0 if base is None else base.long()[:, None])
    taken = (j >= 0) & (j < n)
    if w is not None:
        taken &= ~(w == 0)
    rows = [torch.bincount(j[a:b][taken[a:b]], minlength=n) for a, b in sequences(len(idx), offsets)]
    return torch.stack(rows) if rows else torch.zeros((0, n), dtype=torch.int64)


def balance(logits, counts, *, score="softmax", offsets=None, scale=1.0, dloss=None, add=None):
    """(loss [sequences], the logits' gradient [tokens, n], and for both what 2^-24 relative errors of every share and
    count, less their mean, can move them by)."""
    tokens, n = logits.shape
    p, rest = shares(logits, score)
    grad = torch.zeros((tokens, n), dtype=torch.float64)
    moved = torch.zeros_like(grad)
    loss, shift = [], []
    for s, (a, b) in enumerate(sequences(tokens, offsets)):
        total = int(counts[s].sum())
        if a == b or total == 0:
            loss.append(0.0)
            shift.append(0.0)
            continue
        c, off = counts[s].double(), (counts[s].double() - total / n).abs() + total / n * STEP
        per = scale * n / ((b - a) * total)
        loss.append(float(per * (p[a:b] @ c).sum()))
        shift.append(STEP * (abs(scale) + abs(per) * float((p[a:b] @ off).sum())))
        g = per * (1.0 if dloss is None else float(dloss[s])) * p[a:b] * rest[a:b]
        grad[a:b] = g * (c - (p[a:b] @ c)[:, None])
        moved[a:b] = STEP * g.abs() * (off + (p[a:b] @ off)[:, None])
    if add is not None:
        grad = grad + add.double()
    as64 = lambda v: torch.tensor(v, dtype=torch.float64)  # noqa: E731
    return as64(loss), grad, as64(shift), moved


def row_sums(ops, rows, *, chunk=1, valid=None, chunk_valid=None, scale=1.0, padding=None):
    """(sums [rows, hd], the sums of the magnitudes, terms [rows]) for ops = [(idx [tokens, width], w or None, dout)]."""
    hd = ops[0][2].shape[-1]
    sums, size, terms = (torch.zeros((rows, hd), dtype=torch.float64), torch.zeros((rows, hd), dtype=torch.float64),
                         torch.zeros(rows, dtype=torch.float64))
    for idx, w, dout in ops:
        tokens = len(idx)
        at = torch.arange(tokens)
        until = chunk if valid is None else valid
        live = at % chunk < (torch.full((tokens,), until) if chunk_valid is None else chunk_valid.long().repeat_interleave(chunk))
        weight = torch.ones(idx.shape, dtype=torch.float64) if w is None else w.double()
        idx = idx.long()
        taken = live[:, None] & (idx >= 0) & (idx < rows) & ~(weight == 0)
        if padding is not None:
            taken &= idx != padding
        t, i = taken.nonzero(as_tuple=True)
        values = weight[t, i][:, None] * dout.double()[t] * scale
        sums.index_add_(0, idx[t, i], values)
        size.index_add_(0, idx[t, i], values.abs())
        terms.index_add_(0, idx[t, i], torch.ones(len(t), dtype=torch.float64))
    return sums, size, terms


def close(got: torch.Tensor, want: torch.Tensor, moved: torch.Tensor, what: str, parts: float = 1.0) -> None:
    """got (any type) is want, moved by `parts` times `moved` at most before it was rounded to its type."""
    half = half_step(got.dtype)
    err = (got.cpu().double() - want).abs()
    most = parts * moved
    tiny = 2.0 ** -149 if got.dtype == torch.float32 else 2.0 ** -133  # the least step of the type
    bound = most + half * (want.abs() + most) + tiny
    bad = ~(err <= bound)  # NaN is bad
    if bad.any():
        at = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, at {at}: {float(got.cpu()[at])} for {float(want[at])}, "
                             f"bound {float(bound[at]):.3e}, error {float(err[at]):.3e}")
