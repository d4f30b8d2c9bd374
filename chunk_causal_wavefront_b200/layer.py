"""One transformer layer over a wavefront round, in libwf's kernels.

A pre-norm layer on the residual stream h [S+1][C][hidden] of a round's slots:

    y = norm(h);  q, k, v = y w_qkv^T;  publish;  a = round attention
    h = h + a w_out^T + b_out
    h = h + GELU(norm(h) w_up^T + b_up) w_down^T + b_down

Weights are bf16, or E4M3 rows (8-bit products: "W8A8" beside the 8-bit attention
backends of the appendix's Tables 4-6); the pool is bf16 or FP8 independently of
that. Only the live slots' rows are read and written, so the same object runs
through pipeline fill. Under Wave Parallelism, publish_slot, the deliveries and
attend_slot run one slot on its rank.
"""
from __future__ import annotations

import dataclasses
from typing import Optional, Union

import torch

from . import wf as _wf
from .pool import KVPool
from .rows import E4M3Rows, add_rms_norm, linear, quantize_rows, refuse_gradients, rows_check_status

Weight = Union[torch.Tensor, E4M3Rows]


@dataclasses.dataclass
class LayerWeights:
    """w_qkv [3 hidden, hidden], w_out [hidden, hidden], w_up [ffn, hidden], w_down
    [hidden, ffn]: all bf16 or all E4M3 rows. Norm weights and biases are float32
    vectors; None means ones (norms) or zeros (biases)."""

    w_qkv: Weight
    w_out: Weight
    w_up: Weight
    w_down: Weight
    norm1: Optional[torch.Tensor] = None
    norm2: Optional[torch.Tensor] = None
    b_out: Optional[torch.Tensor] = None
    b_up: Optional[torch.Tensor] = None
    b_down: Optional[torch.Tensor] = None

    def to_e4m3(self) -> "LayerWeights":
        """The same layer with its products in 8 bits."""
        return dataclasses.replace(self, **{n: quantize_rows(getattr(self, n))
                                            for n in ("w_qkv", "w_out", "w_up", "w_down")})


class LayerRound:
    """Runs layers on the rounds of one pool; holds the scratch that a layer needs.

    One object serves all layers of a pool, one call at a time in stream order. The
    calls do not synchronise, so what goes wrong on the device (a missing publication,
    a bounded wait that runs out) is asked for with check_status()."""

    def __init__(self, pool: KVPool, ffn: int, eps: float = 1e-6):
        c = pool.cfg
        if c.dtype == _wf.WF_DTYPE_F32:
            raise ValueError("layers run on bf16 and FP8 pools")
        self.pool, self.eps, self.ffn = pool, eps, ffn
        self.hidden = c.num_heads * c.head_dim
        self.shape = (c.num_stages + 1, c.chunk_tokens, c.num_heads, c.head_dim)
        new = lambda dtype=torch.bfloat16: torch.empty(self.shape, dtype=dtype, device=pool.device)
        self.q_rot, self.att = new(pool.dtype), new()
        self._new, self._qkv = new, None

    # -- rows ---------------------------------------------------------------------------
    def _rows(self, t: torch.Tensor, slot: Optional[int]) -> torch.Tensor:
        """The live slots' rows of a round's buffer, or one slot's."""
        r = t.view(-1, self.hidden)
        chunk = self.shape[1]
        return r[:self.pool.live_rows] if slot is None else r[slot * chunk:(slot + 1) * chunk]

    def _check(self, h: torch.Tensor, w: LayerWeights) -> Optional[str]:
        """Everything that a layer reads, before its first call: the pool's calls take addresses
        without shapes, and a refusal half-way would leave h between two states."""
        if h.dtype != torch.bfloat16 or h.numel() != self.q_rot.numel() or not h.is_contiguous():
            raise ValueError("h must be a contiguous bf16 tensor [S+1][C][hidden]")
        kinds = {isinstance(m, E4M3Rows) for m in (w.w_qkv, w.w_out, w.w_up, w.w_down)}
        if len(kinds) != 1:
            raise ValueError("weights must be all bf16 or all E4M3 rows")
        e4m3 = kinds.pop()
        hidden, ffn = self.hidden, w.w_up.shape[0]
        given = [("h", h)]
        for name, shape in (("w_qkv", (3 * hidden, hidden)), ("w_out", (hidden, hidden)),
                            ("w_up", (ffn, hidden)), ("w_down", (hidden, ffn))):
            m = getattr(w, name)
            if tuple(m.shape) != shape or not (e4m3 or m.dtype == torch.bfloat16):
                raise ValueError(f"{name} must be {list(shape)} in bf16 or E4M3 rows, not {list(m.shape)}")
            c = m.codes if e4m3 else m
            if (c.stride(1) != 1 or c.stride(0) < shape[1] or c.stride(0) * c.element_size() % 16
                    or c.data_ptr() % 16 or (e4m3 and m.scales.data_ptr() % 16)):
                raise ValueError(f"{name} must have contiguous rows that start at multiples of 16 bytes")
            given.append((name, m))
        if ffn % 8:
            raise ValueError(f"the feed-forward's {ffn} features are not a multiple of 8")
        for name, n in (("norm1", hidden), ("norm2", hidden), ("b_out", hidden), ("b_up", ffn), ("b_down", hidden)):
            v = getattr(w, name)
            if v is None:
                continue
            if v.dtype != torch.float32 or v.shape != (n,) or not v.is_contiguous():
                raise ValueError(f"{name} must be a contiguous float32 vector of {n} elements")
            given.append((name, v))
        for name, t in given:
            if t.device != self.q_rot.device:
                raise ValueError(f"{name} is on {t.device}, the pool on {self.q_rot.device}")
        refuse_gradients("layers", *(t for _, t in given))
        return "e4m3" if e4m3 else None

    # -- the two halves around the K/V exchange -------------------------------------------
    def _publish(self, layer: int, h: torch.Tensor, w: LayerWeights, slot: Optional[int], to: Optional[str]) -> None:
        pool, hidden = self.pool, self.hidden
        x = self._rows(h, slot)
        if (slot is None and to is None and pool.cfg.dtype == _wf.WF_DTYPE_BF16
                and hidden % 256 == 0 and pool.cfg.page_tokens == 128):
            # att is free until the attention: it holds the projection's input, of
            # which only the live slots' rows are read.
            add_rms_norm(x, w.norm1, eps=self.eps, out=self._rows(self.att, None))
            pool.project_publish(layer, self.att, w.w_qkv, self.q_rot)
            return
        y = add_rms_norm(x, w.norm1, eps=self.eps, out_dtype=to)
        if self._qkv is None:
            self._qkv = [self._new() for _ in range(3)]
        for i, t in enumerate(self._qkv):
            part = (w.w_qkv.span(i * hidden, (i + 1) * hidden) if to else
                    w.w_qkv[i * hidden:(i + 1) * hidden])
            linear(y, part, out=self._rows(t, slot))
        if slot is None:
            pool.publish(layer, *self._qkv, self.q_rot)
        else:
            pool.publish_slot(layer, slot, *self._qkv, self.q_rot)

    def _attend(self, layer: int, h: torch.Tensor, w: LayerWeights, slot: Optional[int], to: Optional[str]) -> None:
        pool = self.pool
        if slot is None:
            pool.attention(layer, self.q_rot, self.att)
        else:
            pool.attention_slot(layer, slot, self.q_rot, self.att)
        a, r = self._rows(self.att, slot), self._rows(h, slot)
        linear(quantize_rows(a) if to else a, w.w_out, w.b_out, residual=r, out=r)
        y = add_rms_norm(r, w.norm2, eps=self.eps, out_dtype=to)
        u = linear(y, w.w_up, w.b_up, act="gelu", out_dtype=to)
        linear(u, w.w_down, w.b_down, residual=r, out=r)

    # -- calls ------------------------------------------------------------------------------
    def run(self, layer: int, h: torch.Tensor, w: LayerWeights) -> torch.Tensor:
        """The layer on every live slot of the pool's round; updates h in place."""
        to = self._check(h, w)
        self._publish(layer, h, w, None, to)
        self._attend(layer, h, w, None, to)
        return h

    def check_status(self, stream=None) -> int:
        """Synchronise, then return and clear the first error of the calls before: the pool's status,
        or the row operators' of its device."""
        status = self.pool.check_status(stream)
        rows = rows_check_status(self.q_rot.device, stream)
        return status if status != _wf.WF_OK else rows

    def publish_slot(self, layer: int, slot: int, h: torch.Tensor, w: LayerWeights) -> None:
        """Up to the publication of one slot's K/V (its rank delivers them next)."""
        self._publish(layer, h, w, slot, self._check(h, w))

    def attend_slot(self, layer: int, slot: int, h: torch.Tensor, w: LayerWeights) -> torch.Tensor:
        """From the slot's attention on, once the deliveries into this pool have landed."""
        self._attend(layer, h, w, slot, self._check(h, w))
        return h
