"""Host-side decode state of one SDM layer: the memory bank and the number of tokens consumed.

Mirrors ``SDMLayerState`` of the sparse-delta-memory 2.0.0 wheel (cache.py): the state is the bank
(a device tensor updated in place by every decode call) plus a running token count; ``update_``
swaps in a new bank and advances the count, ``reset`` zeroes the bank and the count. ``step`` and
``steps`` advance the state through the C ABI (``sdm_decode_step`` / ``sdm_decode_seq``).

``RoutedLayerState`` is the same for a quantised bank that streams address by logits over their slots:
it chooses the slots (``sdm_route``), advances the bank (``sdm_qdecode_step`` / ``sdm_qdecode_seq``),
reads it without writing (``sdm_qgather``), takes a reading's gradient back to the logits (``sdm_gather_dw``,
``sdm_route_backward``) and to the rows (``sdm_gather_drows``), and balances the choices (``sdm_balance``).
"""

from __future__ import annotations

import torch

from . import quant, routing, sdm


class SDMLayerState:
    """Decode state: ``memory`` [num_slots, head_dim] (bf16 or float32, on the GPU) and ``cache_len``."""

    def __init__(self, memory: torch.Tensor, seq_len: int = 0) -> None:
        self.memory = memory
        self._cache_len = int(seq_len)

    def __getitem__(self, key_idx: int) -> torch.Tensor:
        if key_idx == 0:
            return self.memory
        raise KeyError(key_idx)

    def __len__(self) -> int:
        return 1

    @property
    def cache_len(self) -> int:
        return self._cache_len

    def reset(self) -> None:
        """Zero the bank and the token count."""
        self.memory.zero_()
        self._cache_len = 0

    def update_(self, new_memory: torch.Tensor, seq_len: int = 1) -> "SDMLayerState":
        """Take ``new_memory`` as the bank and count ``seq_len`` more tokens."""
        if self.memory is None:
            raise RuntimeError("the state has no bank")
        self.memory = new_memory.detach()
        self._cache_len += int(seq_len)
        return self

    def step(self, k_idx, k_val, v, beta, g, q_idx, q_val, out=None, stream=None) -> torch.Tensor:
        """One token for every stream (arrays [S, .], beta [S]); returns the readings [S, head_dim]."""
        readings = sdm.decode_step(self.memory, k_idx, k_val, v, beta, g, q_idx, q_val, out=out, stream=stream)
        self._cache_len += 1
        return readings

    def steps(self, k_idx, k_val, v, beta, g, q_idx, q_val, out=None, stream=None) -> torch.Tensor:
        """T tokens for every stream in one launch (time-major arrays [T, S, .], beta [T, S]);
        returns the readings [T, S, head_dim]."""
        readings = sdm.decode_seq(self.memory, k_idx, k_val, v, beta, g, q_idx, q_val, out=out, stream=stream)
        self._cache_len += int(k_idx.shape[0])
        return readings


class RoutedLayerState:
    """Decode state of ``streams`` streams with ``slots`` slots each on a quantised bank: ``memory`` is a
    ``quant.QuantBank`` of streams * slots rows, stream s has the slots from s * slots on.

    Tokens give logits [S, slots] (bfloat16 or float32) over their stream's slots; the ``writes`` best
    of ``k_logits`` are written with the router's weights as k_val, the ``reads`` best of ``q_logits`` are
    read. A slot with a logit of -inf is not chosen while others are left; if it is taken to fill up, its weight is 0,
    so that a write only decays its row. ``router`` holds further arguments of ``routing.route`` (score, bias,
    groups, ...); one set serves both choices."""

    def __init__(self, memory: quant.QuantBank, streams: int, *, writes: int, reads: int, seq_len: int = 0, **router) -> None:
        if streams < 1 or memory.n_slots % streams:
            raise ValueError(f"{memory.n_slots} slots do not divide among {streams} streams")
        for name in ("base", "idx_dtype", "idx", "w", "stream"):
            if name in router:
                raise ValueError(f"{name} is set by the state")
        self.memory, self.streams, self.slots = memory, streams, memory.n_slots // streams
        self.writes, self.reads, self.router = writes, reads, router
        self._cache_len = int(seq_len)
        self._first = torch.arange(streams, device=memory.device) * self.slots

    @property
    def cache_len(self) -> int:
        return self._cache_len

    def reset(self) -> None:
        """Zero the bank and the token count."""
        self.memory.codes.zero_()
        self.memory.scales.zero_()
        self._cache_len = 0

    def load_(self, rows: torch.Tensor, seq_len: int) -> "RoutedLayerState":
        """Take the rows [streams * slots, hd] (bfloat16 or float32) as the bank, after ``seq_len`` tokens."""
        if tuple(rows.shape) != (self.memory.n_slots, self.memory.hd):
            raise ValueError(f"rows must be [{self.memory.n_slots}, {self.memory.hd}], got {tuple(rows.shape)}")
        quant.quantize_rows(self.memory, rows)
        self._cache_len = int(seq_len)
        return self

    def rows(self, dtype=torch.bfloat16) -> torch.Tensor:
        """The bank's rows [streams * slots, hd]."""
        return quant.dequantize_rows(self.memory, dtype=dtype)

    def choose(self, logits: torch.Tensor, k: int):
        """(idx, w) [.., k]: the slots of the bank that logits [.., S, slots] choose, and their weights."""
        if logits.shape[-2:] != (self.streams, self.slots):
            raise ValueError(f"logits must be [.., {self.streams}, {self.slots}], got {tuple(logits.shape)}")
        tokens = logits.shape[:-2].numel()
        first = self._first if tokens == 1 else self._first.repeat(tokens)
        idx, w = routing.route(logits.reshape(-1, self.slots), k, base=first, idx_dtype=torch.int64, **self.router)
        return idx.view(*logits.shape[:-1], k), w.view(*logits.shape[:-1], k)

    def step(self, k_logits, v, beta, g, q_logits, *, out_dtype=torch.bfloat16) -> torch.Tensor:
        """One token for every stream (logits [S, slots], v [S, hd], beta [S], g [S, 1] or
        [S, writes]): written, then read; returns the readings [S, hd]."""
        readings = quant.decode_step(self.memory, *self.choose(k_logits, self.writes), v, beta, g,
                                     *self.choose(q_logits, self.reads), out_dtype=out_dtype)
        self._cache_len += 1
        return readings

    def steps(self, k_logits, v, beta, g, q_logits, *, out_dtype=torch.bfloat16) -> torch.Tensor:
        """T tokens for every stream (time-major arrays [T, S, .], beta [T, S]): two routing launches
        and one decode; returns the readings [T, S, hd], the bits of T calls of ``step``."""
        readings = quant.decode_seq(self.memory, *self.choose(k_logits, self.writes), v, beta, g,
                                    *self.choose(q_logits, self.reads), out_dtype=out_dtype)
        self._cache_len += int(k_logits.shape[0])
        return readings

    def _one_reading(self, q_logits: torch.Tensor) -> None:
        if tuple(q_logits.shape) != (self.streams, self.slots):
            raise ValueError(f"logits must be [{self.streams}, {self.slots}], got {tuple(q_logits.shape)}")

    def read(self, q_logits: torch.Tensor):
        """What logits [S, slots] read, with no write: (readings [S, hd] float32, idx, w)."""
        self._one_reading(q_logits)
        idx, w = self.choose(q_logits, self.reads)
        out, = quant.gather(self.memory, [(idx, w)])
        return out, idx, w

    def read_backward(self, q_logits: torch.Tensor, idx: torch.Tensor, dout: torch.Tensor, w=None) -> torch.Tensor:
        """Gradient of the logits of ``read`` from that of its readings (float32 [S, hd]); ``idx`` and ``w`` as
        it returned them. The choice itself has no gradient, as in any top-k router. Where groups or a bias can
        leave too few slots, the weights tell which only filled up; they are computed again when not given."""
        self._one_reading(q_logits)
        groups = self.router.get("groups", 1)
        if w is None and (self.router.get("bias") is not None or (self.router.get("top_groups") or groups) < groups):
            _, w = self.choose(q_logits, self.reads)
        dw, = quant.gather_dw(self.memory, [(idx, dout)])
        given = {n: self.router[n] for n in ("score", "renorm", "scale") if n in self.router}
        return routing.route_backward(q_logits, idx, dw, base=self._first, w=w, **given)

    def rows_gradient(self, idx: torch.Tensor, w: torch.Tensor, dout: torch.Tensor, *, out=None, accumulate: bool = False) -> torch.Tensor:
        """Gradient [streams * slots, hd] float32 of the rows that ``read`` summed (of the values that their codes stand for),
        from that of its readings (float32 [S, hd]); ``idx`` and ``w`` as it returned them. ``out`` and ``accumulate`` as in
        ``quant.gather_drows``."""
        return quant.gather_drows([(idx, w, dout)], self.memory.n_slots, out=out, accumulate=accumulate)

    def balance(self, logits: torch.Tensor, idx: torch.Tensor, w=None, *, scale: float = 1.0, gradient: bool = False, dloss=None, add=None):
        """The balance loss of choices ``idx`` (and ``w``) [.., S, k] that logits [.., S, slots] made, over the places
        0 .. slots - 1 that the streams' slots share: (loss [1], counts [1, slots]), with ``gradient`` the logits' gradient
        too, added to ``add`` (e.g. what ``read_backward`` returned). ``scale`` and ``dloss`` as in ``routing.balance``."""
        if logits.shape[-2:] != (self.streams, self.slots):
            raise ValueError(f"logits must be [.., {self.streams}, {self.slots}], got {tuple(logits.shape)}")
        if idx.shape[:-1] != logits.shape[:-1]:
            raise ValueError(f"idx must be [.., {self.streams}, k] as the logits, got {tuple(idx.shape)}")
        tokens, k = logits.shape[:-2].numel(), idx.shape[-1]
        first = self._first if tokens == 1 else self._first.repeat(tokens)
        loss, counts, *grad = routing.balance(
            logits.reshape(-1, self.slots), idx.reshape(-1, k), score=self.router.get("score", "softmax"), base=first, scale=scale,
            w=None if w is None else w.reshape(-1, k), gradient=gradient, dloss=dloss, add=None if add is None else add.reshape(-1, self.slots))
        return (loss, counts, grad[0].view(logits.shape)) if gradient else (loss, counts)
