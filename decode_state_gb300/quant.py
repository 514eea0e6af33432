"""Quantised banks: 8-bit and 4-bit memory rows, written, read back, gathered and decoded.

A ``QuantBank`` holds a bank's rows as codes of 8 or 4 bits with one float32 scale for every 32, 64
or 128 columns (layout and rounding: ``include/sdm.h``). ``quantize_rows`` writes rows into its
slots, ``dequantize_rows`` reads them back, ``gather`` sums rows with weights, ``gather_dw`` is the
gradient of those weights (also over bfloat16 and float32 banks), and ``decode_step`` /
``decode_seq`` advance streams on it as ``sdm.decode_step`` / ``sdm.decode_seq`` do on a
floating-point bank. Everything runs in the CUDA library; the native binding checks arguments and
passes pointers. Work goes to the current stream of the bank's device unless ``stream`` is given (a
``torch.cuda.Stream`` or a handle); outputs are then made in that stream's memory, and whoever uses
them on another stream waits for it first, and records its use (``Tensor.record_stream``) before they go.

A user's choice of format: int8 rounds a row's values by about as much as bfloat16 does (1/254 of
the group's largest value at most) and suits rows that are written again and again; fp8 keeps three
bits behind the leading one whatever a value's size, which suits rows with outliers; int4 is for
snapshots that are read (the decode does not take it).
"""

from __future__ import annotations

import torch

from .sdm import binding

FORMATS = {"int8": 2, "fp8": 3, "int4": 4}  # SDM_INT8, SDM_FP8, SDM_INT4


def row_bytes(hd: int, format: str) -> int:
    """Bytes of one row of codes (sdm_quant_row_bytes)."""
    return ((hd + 1) // 2 if format == "int4" else hd) + 15 & ~15


class QuantBank:
    """A quantised bank: ``codes`` [n_slots, row_bytes(hd, format)] uint8 and ``scales``
    [n_slots, ceil(hd / group)] float32, both contiguous on one GPU. It keeps the two tensors and
    nothing else, so a handle over tensors that exist already costs nothing to make."""

    __slots__ = ("codes", "scales", "hd", "group", "format", "_code")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, hd: int, *, group: int = 128, format: str = "int8"):
        if format not in FORMATS:
            raise ValueError(f"format must be one of {sorted(FORMATS)}, got {format!r}")
        if group not in (32, 64, 128):
            raise ValueError(f"group must be 32, 64 or 128 columns, got {group}")
        self.codes, self.scales, self.hd, self.group, self.format = codes, scales, hd, group, format
        self._code = FORMATS[format]
        binding().check_bank(self)

    @property
    def n_slots(self) -> int:
        return self.codes.shape[0]

    @property
    def device(self) -> torch.device:
        return self.codes.device

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
        given = stream
        if stream is not None and not hasattr(stream, "cuda_stream"):  # a handle; 1 is the legacy default stream, as 0 is
            given = torch.cuda.ExternalStream(0 if stream == 1 else stream, rows.device)
        with torch.cuda.stream(given):  # memory that is free for the stream that writes it
            codes = torch.empty((n, row_bytes(hd, format)), dtype=torch.uint8, device=rows.device)
            scales = torch.empty((n, -(-hd // group)), dtype=torch.float32, device=rows.device)
        bank = cls(codes, scales, hd, group=group, format=format)
        quantize_rows(bank, rows, stream=stream)
        return bank


def quantize_rows(bank: QuantBank, rows: torch.Tensor, slots: torch.Tensor | None = None, stream=None) -> QuantBank:
    """Write ``rows`` [n, hd] (bfloat16 or float32; the row stride is free) into the bank's slots
    ``slots`` [n] (distinct; int32 or int64), or into slots 0 .. n - 1 (sdm_quantize_rows)."""
    return binding().rows(True, bank, rows, slots, None, stream)


def dequantize_rows(bank: QuantBank, slots: torch.Tensor | None = None, *, dtype=torch.bfloat16, out=None,
                    stream=None) -> torch.Tensor:
    """The rows in ``slots`` [n] (repeats allowed), or all rows, as bfloat16 or float32 [n, hd]
    (sdm_dequantize_rows); ``out`` gives the tensor to write (its row stride is free)."""
    return binding().rows(False, bank, out, slots, dtype, stream)


def gather(bank: QuantBank, ops, *, chunk: int = 1, valid: int | None = None, chunk_valid=None, outs=None,
           stream=None) -> list:
    """Weighted sums of quantised rows (sdm_qgather): for ``ops = [(idx, w), ...]`` (one or two;
    idx and w [tokens, width], w bfloat16 or float32) the list of [tokens, hd] float32 sums.
    ``chunk``, ``valid`` and ``chunk_valid`` mark padding tokens as in ``sdm.gather``; an entry whose
    index is outside the bank is skipped.

    From 4096 tokens and operands on, a weight times its row's scale keeps all its bits down to 2^-22 of the
    largest of up to 32 neighbouring entries, and nothing below 2^-46 of it: a small entry beside a large one
    loses bits that a float32 sum would keep where the large one's code is 0."""
    return binding().gather(bank, ops, chunk, valid, chunk_valid, None, outs, stream, False)


def gather_dw(bank, ops, *, chunk: int = 1, valid: int | None = None, chunk_valid=None, dtype=torch.float32, dws=None,
              stream=None) -> list:
    """Gradient of a gather's weights (sdm_gather_dw): ``bank`` is a QuantBank, or the [n_slots, hd]
    bfloat16 or float32 bank of ``sdm.gather``; ``ops = [(idx, dout), ...]`` with idx [tokens, width]
    and the gradient dout [tokens, hd] (float32) of that operand's output. Returns the list of
    [tokens, width] gradients in ``dtype`` (bfloat16 or float32), zero for an index outside the bank. From
    4096 tokens and operands on, dout enters relative to the largest of its columns as the weights of
    ``gather`` do (not over a float32 bank)."""
    return binding().gather(bank, ops, chunk, valid, chunk_valid, dtype, dws, stream, True)


def decode_step(bank: QuantBank, k_idx, k_val, v, beta, g, q_idx, q_val, out=None, *, out_dtype=torch.bfloat16,
                stream=None) -> torch.Tensor:
    """One write-then-read token for every stream on a quantised bank (sdm_qdecode_step): arrays
    [S, .], beta [S]; the bank is updated in place; returns the readings [S, hd] in ``out_dtype``."""
    return binding().decode(bank, k_idx, k_val, v, beta, g, q_idx, q_val, out, out_dtype, 1, False, stream)


def decode_seq(bank: QuantBank, k_idx, k_val, v, beta, g, q_idx, q_val, out=None, *, out_dtype=torch.bfloat16,
               stream_major: bool = False, stream=None) -> torch.Tensor:
    """T tokens for every stream in one launch (sdm_qdecode_seq): time-major arrays [T, S, .], beta
    [T, S] (``stream_major``: [S, T, .]); returns the readings in the same layout."""
    return binding().decode(bank, k_idx, k_val, v, beta, g, q_idx, q_val, out, out_dtype, 2, stream_major, stream)
