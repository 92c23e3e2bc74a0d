"""Prompt-side runner: a chunk of new tokens of a ragged batch through one layer.

The dense form, for a prompt, a context no longer than the Top-K, or a verification
of draft tokens: rotary positions on the queries, the new tokens' rows normed,
rotated, quantized and appended to the FP4 cache, then attention of the chunk
over every visible position of it.  Three library calls; no arithmetic here.

Attention reads FP4 rows alone.  The decode step (``step.py``) joins them with the
exact bf16 rows of the newest tokens where its layer has a window (``swa`` > 0): the
two are the same function only for a layer without one (``swa`` 0) whose Top-K set
holds every position.  ``entry`` keeps the exact rows for a decode step's window.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import csa2


@dataclass
class ChunkBuffers:
    """Device tensors of one layer's chunk (all on the same CUDA device)."""
    dims: csa2.Dims
    batch: int
    rope: csa2.Rope
    # cache
    kv_codes: torch.Tensor          # uint8 [rows, 256]
    kv_scales: torch.Tensor         # uint8 [rows, 32]
    kv_rope: torch.Tensor           # bf16  [rows, 64]
    page_table: torch.Tensor | None
    ctx_len: torch.Tensor           # int32 [B]: contexts, the chunk's tokens included
    # the chunk: the new tokens of all sequences, packed
    q_start: torch.Tensor           # int32 [B + 1]
    q: torch.Tensor                 # bf16 [total, H, 576]; its last 64 channels are rotated in place
    x: torch.Tensor                 # bf16 [total, 576] projections (latent | rotary part) of the new tokens
    pos: torch.Tensor               # int32 [total] positions
    dst_rows: torch.Tensor          # int64 [total] cache rows (negative: none, a padding token; see cache_rows)
    scale: float
    norm_w: torch.Tensor | None = None   # bf16 [512]
    eps: float = 1e-6
    window: int = 0
    entry: torch.Tensor | None = None    # bf16 [total, 576]: also receives the exact rows, for a later decode step's window
    # outputs
    out: torch.Tensor = None        # bf16 [total, H, 512]
    lse: torch.Tensor = None        # fp32 [total, H]
    ws: torch.Tensor = None

    def allocate_outputs(self):
        total, h, dev = self.q.shape[0], self.dims.heads, self.q.device
        self.out = torch.empty((total, h, csa2.LATENT), dtype=torch.bfloat16, device=dev)
        self.lse = torch.empty((total, h), dtype=torch.float32, device=dev)
        self.ws = csa2.alloc_dense_attn_workspace(self.dims, self.batch, total, device=dev)
        return self


def cache_rows(ctx_len, q_start, page_table=None, max_ctx: int = 0, total: int | None = None):
    """Positions (int32 [total]) and cache rows (int64 [total]) of a chunk's tokens.

    ctx_len: contexts with the chunk included; q_start: as in ChunkBuffers; total: packed
    tokens, padding included (None: q_start[-1]); max_ctx: rows of a sequence in a cache
    without a page table (needed for more than one).  Token i of sequence b, of n, stands at
    position ctx_len[b] - n + i; a position below 0 (more tokens than context) or behind the
    sequence's rows (its pages, max_ctx) has no row, nor has a padding token, before q_start[0]
    or from q_start[-1] on (its position is 0)."""
    starts, batch, dev = q_start.long(), ctx_len.numel(), q_start.device
    csa2._need("cache_rows", starts.numel() == batch + 1 and (page_table is not None or batch <= 1 or max_ctx > 0))
    t = torch.arange(int(starts[-1]) if total is None else total, device=dev)
    room = page_table.shape[1] * csa2.PAGE if page_table is not None else max_ctx if max_ctx > 0 else 1 << 31
    if batch == 0 or room == 0:
        return torch.zeros_like(t, dtype=torch.int32), torch.full_like(t, -1)
    b = torch.searchsorted(starts[1:].contiguous(), t, right=True).clamp(max=batch - 1)
    own = (t >= starts[b]) & (t < starts[b + 1])
    pos = torch.where(own, ctx_len.long()[b] - (starts[b + 1] - t), torch.zeros_like(t))
    at = pos.clamp(min=0, max=room - 1)
    if page_table is None:
        rows = b * max_ctx + at
    else:
        rows = page_table.long()[b, at // csa2.PAGE] * csa2.PAGE + at % csa2.PAGE
    return pos.to(torch.int32), torch.where(own & (pos == at), rows, torch.full_like(rows, -1))


def run_chunk(cb: ChunkBuffers, stream=None):
    """Enqueue the chunk: three library calls in order on one stream."""
    csa2.csa2_rope_apply(cb.rope, cb.q, cb.pos, y=cb.q, offset=csa2.LATENT, stream=stream)
    csa2.csa2_kv_append(cb.rope, cb.x, cb.pos, cb.dst_rows, cb.kv_codes, cb.kv_scales, cb.kv_rope, norm_w=cb.norm_w,
                        eps=cb.eps, entry=cb.entry, stream=stream)
    csa2.csa2_dense_attn_chunk(cb.dims, cb.batch, cb.q, cb.q_start, cb.kv_codes, cb.kv_scales, cb.kv_rope, cb.page_table,
                               cb.ctx_len, cb.scale, cb.out, cb.lse, cb.ws, window=cb.window, stream=stream)
