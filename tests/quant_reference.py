"""Plain implementations of the quantised-bank and routing operators, on the CPU.

Quantisation is defined in float32 (a division, a product and a rounding), so its reference is
float32 numpy and is met bit for bit; all sums are float64.
"""

from __future__ import annotations

import numpy as np

LEVELS = {"int8": 127.0, "fp8": 448.0, "int4": 7.0}
EPS = 2.0 ** -24  # half a unit in the last place of a float32 below 1: one rounding's relative error


def e4m3_table() -> np.ndarray:
    """Values of the 256 codes of 4 exponent and 3 mantissa bits (float64)."""
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    mag = np.where(e > 0, (1 + m / 8) * 2.0 ** (e - 7), m / 8 * 2.0 ** -6)
    mag[(e == 15) & (m == 7)] = np.nan
    return np.where(b & 128, -mag, mag)


def e4m3_round(y: np.ndarray) -> np.ndarray:
    """Codes of float32 values of magnitude <= 448 (one rounding above it included), nearest even."""
    table = e4m3_table()[:127]  # 0 .. 448
    mag = np.minimum(np.abs(y).astype(np.float64), 448.0)
    hi = np.searchsorted(table, mag).clip(1, 126)
    lo = hi - 1
    dl, dh = mag - table[lo], table[hi] - mag
    code = np.where(dl < dh, lo, np.where(dl > dh, hi, np.where(lo % 2 == 0, lo, hi)))
    return (code | np.where(np.signbit(y), 128, 0)).astype(np.uint8)


def quantise(x: np.ndarray, group: int, fmt: str):
    """float32 rows [n, hd] -> (codes [n, row_bytes] uint8, scales [n, groups] float32)."""
    n, hd = x.shape
    groups = -(-hd // group)
    level = np.float32(LEVELS[fmt])
    scales = np.zeros((n, groups), np.float32)
    q = np.zeros((n, hd), np.float32)
    with np.errstate(all="ignore"):
        for i in range(groups):
            part = x[:, i * group:(i + 1) * group].astype(np.float32)
            top = np.abs(part).max(axis=1)
            bad = ~np.isfinite(part).all(axis=1)
            zero = ~bad & (top < np.float32(2.0 ** -100))
            scales[:, i] = np.where(bad, np.nan, np.where(zero, 0, top / level))
            inv = (level / np.where(bad | zero, 1, top)).astype(np.float32)
            q[:, i * group:(i + 1) * group] = np.where((bad | zero)[:, None], 0, part * inv[:, None])
    if fmt == "fp8":
        codes = e4m3_round(q)
    else:
        codes = np.rint(q).astype(np.int32)
    if fmt == "int4":
        codes = np.pad(codes, ((0, 0), (0, hd % 2)))
        codes = (codes[:, 0::2] & 15) | ((codes[:, 1::2] & 15) << 4)
    codes = codes.astype(np.uint8) if fmt != "int8" else codes.astype(np.int8).view(np.uint8)
    return np.pad(codes, ((0, 0), (0, -codes.shape[1] % 16))), scales


def values(codes: np.ndarray, scales: np.ndarray, hd: int, group: int, fmt: str) -> np.ndarray:
    """float64 rows of codes [..., row_bytes] and scales [..., groups]."""
    if fmt == "fp8":
        y = e4m3_table()[codes]
    elif fmt == "int8":
        y = codes.view(np.int8).astype(np.float64)
    else:
        nib = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1).astype(np.int64)
        y = np.where(nib >= 8, nib - 16, nib).astype(np.float64)
    return y[..., :hd] * scales.astype(np.float64)[..., np.arange(hd) // group]


# ---------------------------------------------------------------- routing

def scores(x: np.ndarray, kind: str) -> np.ndarray:
    """float64 scores of logits [t, n]; masked entries (-inf, NaN) have 0."""
    x = np.where(np.isnan(x), -np.inf, x.astype(np.float64))
    with np.errstate(all="ignore"):
        if kind == "sigmoid":
            return 1 / (1 + np.exp(-x))
        m = x.max(axis=1, keepdims=True)
        e = np.where(x == m, 1.0, np.exp(x - m))
        e[x == -np.inf] = 0
        s = e.sum(axis=1, keepdims=True)
        return np.where(s > 0, e / np.where(s > 0, s, 1), 0)


def ranks(x: np.ndarray, kind: str, bias=None) -> np.ndarray:
    """float64 ranks; -inf for masked entries."""
    s = scores(x, kind)
    r = s + bias.astype(np.float64) if bias is not None else (s if kind == "sigmoid" else x.astype(np.float64))
    return np.where(np.isnan(x) | (x == -np.inf) | np.isnan(r), -np.inf, r)


def drop_groups(r: np.ndarray, x: np.ndarray, kind: str, bias, groups: int, top_groups: int, group_top: int):
    """Ranks with the entries of the groups that do not stay masked."""
    if groups == 1 or top_groups == groups:
        return r
    by = r.reshape(len(r), groups, -1)
    judged = by
    if group_top == 2 and kind == "softmax" and bias is None:
        judged = np.where(by == -np.inf, -np.inf, scores(x, kind).reshape(by.shape))
    best = -np.sort(-judged, axis=2)[..., :group_top]
    score = np.where(best[..., 0] == -np.inf, -np.inf, np.where(best == -np.inf, 0, best).sum(axis=2))
    order = np.argsort(-score, axis=1, kind="stable")[:, :top_groups]
    keep = np.zeros(score.shape, bool)
    np.put_along_axis(keep, order, True, axis=1)
    return np.where(keep[..., None], by, -np.inf).reshape(r.shape)


def route(x, k, kind, bias=None, groups=1, top_groups=None, group_top=1, renorm=True, scale=1.0):
    r = drop_groups(ranks(x, kind, bias), x, kind, bias, groups, top_groups or groups, group_top)
    idx = np.argsort(-r, axis=1, kind="stable")[:, :k]
    w = np.where(np.take_along_axis(r, idx, 1) == -np.inf, 0, np.take_along_axis(scores(x, kind), idx, 1))
    if renorm:
        s = w.sum(axis=1, keepdims=True)
        w = np.where(s > 0, w / np.where(s > 0, s, 1), 0)
    return idx, w * scale


def weights_of(x, idx, kind, renorm, scale):
    """float64 weights of given entries: what the gradient differentiates."""
    w = np.take_along_axis(scores(x, kind), idx, 1)
    return w * scale / (w.sum(axis=1, keepdims=True) if renorm else 1)


def route_backward(x, idx, dw, kind, renorm, scale):
    """(float64 gradient of the logits, the sum of the magnitudes that make each of them up)."""
    s = scores(x, kind)
    c = np.take_along_axis(s, idx, 1)
    u = dw.astype(np.float64) * scale
    size = np.abs(u)
    if renorm:
        total = c.sum(axis=1, keepdims=True)
        total = np.where(total > 0, total, np.inf)
        w = c / total
        size = (size + (size * w).sum(axis=1, keepdims=True)) / total
        u = (u - (u * w).sum(axis=1, keepdims=True)) / total
    full, fsize = np.zeros(s.shape), np.zeros(s.shape)
    np.put_along_axis(full, idx, u, 1)
    np.put_along_axis(fsize, idx, size, 1)
    if kind == "sigmoid":
        return full * s * (1 - s), fsize * s
    mean = (u * c).sum(axis=1, keepdims=True)
    msize = (size * c).sum(axis=1, keepdims=True)
    return s * (full - mean), s * (fsize + msize)
