"""Quantised banks: 8-bit and 4-bit memory rows, written, read back, gathered and decoded.

A ``QuantBank`` holds a bank's rows as codes of 8 or 4 bits with one float32 scale for every 32, 64
or 128 columns (layout and rounding: ``include/sdm.h``). ``quantize_rows`` writes rows into its
slots, ``dequantize_rows`` reads them back, ``gather`` sums rows with weights, ``gather_dw`` is the
gradient of those weights (also over bfloat16 and float32 banks), and ``decode_step`` /
``decode_seq`` advance streams on it as ``sdm.decode_step`` / ``sdm.decode_seq`` do on a
floating-point bank. Everything runs in the CUDA library; these functions check their arguments and
pass pointers. Work goes to the current stream of the bank's device unless ``stream`` is given.

A user's choice of format: int8 rounds a row's values by about as much as bfloat16 does (1/254 of
the group's largest value at most) and suits rows that are written again and again; fp8 keeps three
bits behind the leading one whatever a value's size, which suits rows with outliers; int4 is for
snapshots that are read (the decode does not take it).
"""

from __future__ import annotations

import ctypes

import torch

from . import sdm
from .sdm import _BANK_CODES, _IDX_CODES, _check, _need, _shape, _stream_handle

FORMATS = {"int8": 2, "fp8": 3, "int4": 4}  # SDM_INT8, SDM_FP8, SDM_INT4


def row_bytes(hd: int, format: str) -> int:
    """Bytes of one row of codes (sdm_quant_row_bytes)."""
    return ((hd + 1) // 2 if format == "int4" else hd) + 15 & ~15


class QuantBank:
    """A quantised bank: ``codes`` [n_slots, row_bytes(hd, format)] uint8 and ``scales``
    [n_slots, ceil(hd / group)] float32, both contiguous on one GPU. It keeps the two tensors and
    nothing else, so a handle over tensors that exist already costs nothing to make."""

    __slots__ = ("codes", "scales", "hd", "group", "format", "n_slots", "device", "_args")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, hd: int, *, group: int = 128, format: str = "int8"):
        if format not in FORMATS:
            raise ValueError(f"format must be one of {sorted(FORMATS)}, got {format!r}")
        if group not in (32, 64, 128):
            raise ValueError(f"group must be 32, 64 or 128 columns, got {group}")
        if codes.dtype != torch.uint8 or scales.dtype != torch.float32:
            raise TypeError(f"codes must be uint8 and scales float32, got {codes.dtype}, {scales.dtype}")
        n_slots = codes.shape[0]
        _shape(codes, "codes", (n_slots, row_bytes(hd, format)))
        _shape(scales, "scales", (n_slots, -(-hd // group)))
        device = codes.device
        _need(codes, "codes", device)
        _need(scales, "scales", device)
        self.codes, self.scales, self.hd, self.group, self.format = codes, scales, hd, group, format
        self.n_slots, self.device = n_slots, device
        self._args = (codes.data_ptr(), scales.data_ptr(), n_slots, hd, group, FORMATS[format])

    @classmethod
    def zeros(cls, n_slots: int, hd: int, *, group: int = 128, format: str = "int8", device="cuda") -> "QuantBank":
        """A bank of zero rows."""
        codes = torch.zeros((n_slots, row_bytes(hd, format)), dtype=torch.uint8, device=device)
        scales = torch.zeros((n_slots, -(-hd // group)), dtype=torch.float32, device=device)
        return cls(codes, scales, hd, group=group, format=format)

    @classmethod
    def from_rows(cls, rows: torch.Tensor, *, group: int = 128, format: str = "int8", stream=None) -> "QuantBank":
        """The bank [n_slots, hd] (bfloat16 or float32) quantised, e.g. to go on decoding on 8 bits."""
        n, hd = rows.shape
        codes = torch.empty((n, row_bytes(hd, format)), dtype=torch.uint8, device=rows.device)
        scales = torch.empty((n, -(-hd // group)), dtype=torch.float32, device=rows.device)
        bank = cls(codes, scales, hd, group=group, format=format)
        quantize_rows(bank, rows, stream=stream)
        return bank


def _rows_args(bank: QuantBank, rows: torch.Tensor, slots, name: str):
    if rows.dtype not in _BANK_CODES:
        raise TypeError(f"{name} must be bfloat16 or float32, got {rows.dtype}")
    if rows.dim() != 2 or rows.shape[1] != bank.hd:
        raise ValueError(f"{name} must be [n, {bank.hd}], got {tuple(rows.shape)}")
    if rows.device != bank.device:
        raise ValueError(f"{name} must be a CUDA tensor on {bank.device}, got {rows.device}")
    n = rows.shape[0]
    if n > 1 and rows.stride(0) < bank.hd or bank.hd > 1 and rows.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous columns and rows that do not overlap")
    if slots is None:
        if n > bank.n_slots:
            raise ValueError(f"{n} rows do not fit a bank of {bank.n_slots} slots")
        return n, max(rows.stride(0), bank.hd), None, 0
    _need(slots, "slots", bank.device)
    if slots.dtype not in _IDX_CODES:
        raise TypeError(f"slots must be int32 or int64, got {slots.dtype}")
    _shape(slots, "slots", (n,))
    return n, max(rows.stride(0), bank.hd), slots.data_ptr(), _IDX_CODES[slots.dtype]


def quantize_rows(bank: QuantBank, rows: torch.Tensor, slots: torch.Tensor | None = None, stream=None) -> QuantBank:
    """Write ``rows`` [n, hd] (bfloat16 or float32; the row stride is free) into the bank's slots
    ``slots`` [n] (distinct; int32 or int64), or into slots 0 .. n - 1 (sdm_quantize_rows)."""
    n, stride, slot_ptr, it = _rows_args(bank, rows, slots, "rows")
    rc = sdm.library().sdm_quantize_rows(*bank._args, rows.data_ptr(), stride, _BANK_CODES[rows.dtype], slot_ptr, it, n,
                                         _stream_handle(stream, bank.device))
    _check("sdm_quantize_rows", rc)
    return bank


def dequantize_rows(bank: QuantBank, slots: torch.Tensor | None = None, *, dtype=torch.bfloat16, out=None,
                    stream=None) -> torch.Tensor:
    """The rows in ``slots`` [n] (repeats allowed), or all rows, as bfloat16 or float32 [n, hd]
    (sdm_dequantize_rows); ``out`` gives the tensor to write (its row stride is free)."""
    if out is None:
        out = torch.empty((bank.n_slots if slots is None else slots.shape[0], bank.hd), dtype=dtype, device=bank.device)
    n, stride, slot_ptr, it = _rows_args(bank, out, slots, "out")
    rc = sdm.library().sdm_dequantize_rows(*bank._args, out.data_ptr(), stride, _BANK_CODES[out.dtype], slot_ptr, it, n,
                                           _stream_handle(stream, bank.device))
    _check("sdm_dequantize_rows", rc)
    return out


def _operands(ops, dev, second: str):
    """Checks shared by the gather and the weights' gradient; returns (tokens, index dtype)."""
    if len(ops) not in (1, 2):
        raise ValueError("gather takes one or two operands")
    tokens, it = ops[0][0].shape[0], ops[0][0].dtype
    if it not in _IDX_CODES:
        raise TypeError("indices must be int32 or int64")
    for o, (idx, x) in enumerate(ops):
        _need(idx, f"idx[{o}]", dev)
        _need(x, f"{second}[{o}]", dev)
        if idx.dtype != it or x.dtype != ops[0][1].dtype:
            raise TypeError(f"both operands must share the index dtype and the dtype of {second}")
        if idx.dim() != 2 or idx.shape[0] != tokens:
            raise ValueError(f"idx[{o}] must be [tokens, width]")
    return tokens, it


def _valid(chunk_valid, valid, chunk, tokens, dev):
    if chunk_valid is None:
        return chunk if valid is None else valid, None
    _need(chunk_valid, "chunk_valid", dev)
    if chunk_valid.dtype != torch.int32:
        raise TypeError("chunk_valid must be int32")
    if tokens % chunk == 0:
        _shape(chunk_valid, "chunk_valid", (tokens // chunk,))
    return 0, chunk_valid.data_ptr()


_PTR2, _INT2 = ctypes.c_void_p * 2, ctypes.c_int * 2


def _pointers(tensors):
    return _PTR2(*[t.data_ptr() for t in tensors])


def gather(bank: QuantBank, ops, *, chunk: int = 1, valid: int | None = None, chunk_valid=None, outs=None,
           stream=None) -> list:
    """Weighted sums of quantised rows (sdm_qgather): for ``ops = [(idx, w), ...]`` (one or two;
    idx and w [tokens, width], w bfloat16 or float32) the list of [tokens, hd] float32 sums.
    ``chunk``, ``valid`` and ``chunk_valid`` mark padding tokens as in ``sdm.gather``."""
    dev = bank.device
    tokens, it = _operands(ops, dev, "w")
    wt = ops[0][1].dtype
    if wt not in _BANK_CODES:
        raise TypeError(f"weights must be bfloat16 or float32, got {wt}")
    for o, (idx, w) in enumerate(ops):
        _shape(w, f"w[{o}]", idx.shape)
    if outs is None:
        outs = [torch.empty((tokens, bank.hd), dtype=torch.float32, device=dev) for _ in ops]
    if len(outs) != len(ops):
        raise ValueError("outs must have a tensor for each operand")
    for o, out in enumerate(outs):
        _need(out, f"out[{o}]", dev)
        sdm._f32(out, f"out[{o}]")
        _shape(out, f"out[{o}]", (tokens, bank.hd))
    valid, cv = _valid(chunk_valid, valid, chunk, tokens, dev)
    rc = sdm.library().sdm_qgather(*bank._args, len(ops), _pointers([op[0] for op in ops]),
                                   _pointers([op[1] for op in ops]), _pointers(outs),
                                   _INT2(*[op[0].shape[1] for op in ops]), _IDX_CODES[it], _BANK_CODES[wt], tokens,
                                   chunk, valid, cv, _stream_handle(stream, dev))
    _check("sdm_qgather", rc)
    return outs


def gather_dw(bank, ops, *, chunk: int = 1, valid: int | None = None, chunk_valid=None, dtype=torch.float32, dws=None,
              stream=None) -> list:
    """Gradient of a gather's weights (sdm_gather_dw): ``bank`` is a QuantBank, or the [n_slots, hd]
    bfloat16 or float32 bank of ``sdm.gather``; ``ops = [(idx, dout), ...]`` with idx [tokens, width]
    and the gradient dout [tokens, hd] (float32) of that operand's output. Returns the list of
    [tokens, width] gradients in ``dtype`` (bfloat16 or float32)."""
    if isinstance(bank, QuantBank):
        dev, hd, args = bank.device, bank.hd, bank._args
    else:
        if bank.dtype not in _BANK_CODES or bank.dim() != 2:
            raise TypeError("bank must be a QuantBank or a [n_slots, head_dim] bfloat16 or float32 tensor")
        dev, hd = bank.device, bank.shape[1]
        _need(bank, "bank", dev)
        args = (bank.data_ptr(), None, bank.shape[0], hd, 0, _BANK_CODES[bank.dtype])
    tokens, it = _operands(ops, dev, "dout")
    for o, (_, dout) in enumerate(ops):
        sdm._f32(dout, f"dout[{o}]")
        _shape(dout, f"dout[{o}]", (tokens, hd))
    if dws is None:
        dws = [torch.empty(op[0].shape, dtype=dtype, device=dev) for op in ops]
    if len(dws) != len(ops):
        raise ValueError("dws must have a tensor for each operand")
    dt = dws[0].dtype
    if dt not in _BANK_CODES:
        raise TypeError(f"the gradients must be bfloat16 or float32, got {dt}")
    for o, dw in enumerate(dws):
        _need(dw, f"dw[{o}]", dev)
        _shape(dw, f"dw[{o}]", ops[o][0].shape)
        if dw.dtype != dt:
            raise TypeError("both gradients must share a dtype")
    valid, cv = _valid(chunk_valid, valid, chunk, tokens, dev)
    rc = sdm.library().sdm_gather_dw(*args, len(ops), _pointers([op[0] for op in ops]), _pointers([op[1] for op in ops]),
                                     _pointers(dws), _INT2(*[op[0].shape[1] for op in ops]), _IDX_CODES[it],
                                     _BANK_CODES[dt], tokens, chunk, valid, cv, _stream_handle(stream, dev))
    _check("sdm_gather_dw", rc)
    return dws


def _decode_args(bank: QuantBank, k_idx, k_val, v, beta, g, q_idx, q_val, out, out_dtype, lead: tuple):
    if bank.format == "int4":
        raise ValueError("the decode takes int8 and fp8 banks")
    dev, hd = bank.device, bank.hd
    if k_idx.dtype not in _IDX_CODES or q_idx.dtype != k_idx.dtype:
        raise TypeError(f"k_idx and q_idx must share one dtype, int32 or int64; got {k_idx.dtype}, {q_idx.dtype}")
    W, R, G = k_idx.shape[-1], q_idx.shape[-1], g.shape[-1]
    for name, t, shp in (("k_idx", k_idx, (*lead, W)), ("k_val", k_val, (*lead, W)), ("v", v, (*lead, hd)),
                         ("beta", beta, lead), ("g", g, (*lead, G)), ("q_idx", q_idx, (*lead, R)),
                         ("q_val", q_val, (*lead, R))):
        _need(t, name, dev)
        _shape(t, name, shp)
    for name, t in (("k_val", k_val), ("v", v), ("beta", beta), ("g", g), ("q_val", q_val)):
        sdm._f32(t, name)
    if out is None:
        out = torch.empty((*lead, hd), dtype=out_dtype, device=dev)
    _need(out, "out", dev)
    _shape(out, "out", (*lead, hd))
    if out.dtype not in _BANK_CODES:
        raise TypeError(f"readings must be bfloat16 or float32, got {out.dtype}")
    return out, (k_idx.data_ptr(), k_val.data_ptr(), v.data_ptr(), beta.data_ptr(), g.data_ptr(), q_idx.data_ptr(),
                 q_val.data_ptr(), out.data_ptr()), W, R, G


def decode_step(bank: QuantBank, k_idx, k_val, v, beta, g, q_idx, q_val, out=None, *, out_dtype=torch.bfloat16,
                stream=None) -> torch.Tensor:
    """One write-then-read token for every stream on a quantised bank (sdm_qdecode_step): arrays
    [S, .], beta [S]; the bank is updated in place; returns the readings [S, hd] in ``out_dtype``."""
    S = k_idx.shape[0]
    out, ptrs, W, R, G = _decode_args(bank, k_idx, k_val, v, beta, g, q_idx, q_val, out, out_dtype, (S,))
    codes, scales, n_slots, hd, group, fmt = bank._args
    rc = sdm.library().sdm_qdecode_step(codes, scales, n_slots, *ptrs, S, hd, group, fmt, W, R, G,
                                        _IDX_CODES[k_idx.dtype], _BANK_CODES[out.dtype],
                                        _stream_handle(stream, bank.device))
    _check("sdm_qdecode_step", rc)
    return out


def decode_seq(bank: QuantBank, k_idx, k_val, v, beta, g, q_idx, q_val, out=None, *, out_dtype=torch.bfloat16,
               stream_major: bool = False, stream=None) -> torch.Tensor:
    """T tokens for every stream in one launch (sdm_qdecode_seq): time-major arrays [T, S, .], beta
    [T, S] (``stream_major``: [S, T, .]); returns the readings in the same layout."""
    lead = tuple(k_idx.shape[:2])
    S, T = lead if stream_major else lead[::-1]
    out, ptrs, W, R, G = _decode_args(bank, k_idx, k_val, v, beta, g, q_idx, q_val, out, out_dtype, lead)
    codes, scales, n_slots, hd, group, fmt = bank._args
    rc = sdm.library().sdm_qdecode_seq(codes, scales, n_slots, *ptrs, S, hd, group, fmt, W, R, G, T,
                                       _IDX_CODES[k_idx.dtype], _BANK_CODES[out.dtype],
                                       sdm.SDM_STREAM_MAJOR if stream_major else 0, _stream_handle(stream, bank.device))
    _check("sdm_qdecode_seq", rc)
    return out
