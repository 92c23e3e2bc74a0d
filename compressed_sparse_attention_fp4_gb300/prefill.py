"""Prompt-side runner: a chunk of new tokens of a ragged batch through one layer.

The dense form, for a prompt, a context no longer than the Top-K, or a verification
of draft tokens: rotary positions on the queries, the new tokens' rows normed,
rotated, quantized and appended to the FP4 cache, then attention of the chunk
over every visible position of it.  With `exact` and `keys`, what a layer has beside
that: the window of exact rows, joined in one softmax, and the indexer's keys.
Library calls in order; no arithmetic here.

The decode step (``step.py``) attends to the FP4 rows of its Top-K set and, where its
layer has a window (``swa`` > 0), to the exact bf16 rows of the newest tokens.  The two are
the same function for a Top-K set that holds every position, with `exact` of a window of
``swa`` positions, or without it for ``swa`` 0.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import csa2


@dataclass
class ExactRows:
    """A layer's window over exact bf16 rows: where the chunk's rows go, and what it reads of earlier ones."""
    kv: torch.Tensor                # bf16 [rows, 576], written and read
    dst_rows: torch.Tensor          # int64 [total] its rows for the new tokens (cache_rows)
    window: int                     # positions that a token sees, its own among them
    sinks: int = 0                  # first positions that stay visible
    # of this cache (heads, max_ctx, pages); None: the chunk's, and its page table where none is given here
    dims: csa2.Dims | None = None
    page_table: torch.Tensor | None = None
    # the same rows for a decode step's window, in place (window_rows); both or neither
    swa: torch.Tensor | None = None          # bf16 [B, W, 576]
    swa_rows: torch.Tensor | None = None     # int64 [total]
    ws: torch.Tensor = None
    # positions after which the pages of a sequence come round, whole pages (0: they do not).  All rows of a chunk are
    # written before its attention, so a ring holds what its first token sees and all new tokens: run_chunk
    # refuses a chunk of more than ring - window + 1 tokens of a sequence.
    ring: int = 0


@dataclass
class IndexerKeys:
    """The new tokens' indexer keys: written to the cache rows of their FP4 rows."""
    x: torch.Tensor                 # bf16 [total, 128], fp32 [total, 64] for IDXK_F32: projections
    idx_k: torch.Tensor             # the indexer-K buffer
    cache_rows: int                 # its rows
    kind: int = csa2.IDXK_E4M3
    rope: csa2.Rope | None = None   # on channels [offset, offset + rope.rot)
    offset: int = 0
    norm: int = csa2.IDX_NORM_NONE
    norm_w: torch.Tensor | None = None
    norm_b: torch.Tensor | None = None
    eps: float = 1e-6


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
    # what else the layer has
    exact: ExactRows | None = None
    keys: IndexerKeys | None = None
    longest: int = 0                     # most new tokens of a sequence (0: they may all be one's); for rings of pages

    def allocate_outputs(self):
        total, h, dev = self.q.shape[0], self.dims.heads, self.q.device
        self.out = torch.empty((total, h, csa2.LATENT), dtype=torch.bfloat16, device=dev)
        self.lse = torch.empty((total, h), dtype=torch.float32, device=dev)
        self.ws = csa2.alloc_dense_attn_workspace(self.dims, self.batch, total, device=dev)
        if self.exact is not None:
            self.exact.ws = csa2.alloc_window_attn_workspace(self.exact.dims or self.dims, self.batch, total, device=dev)
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


def window_rows(ctx_len, q_start, window: int, total: int | None = None):
    """Rows (int64 [total]) of a chunk's tokens in a decode step's window [B, window, 576]: position t of
    sequence b at row b * window + t % window.  Tokens that newer ones of the chunk push out of the
    window have none (of several query tokens, decode_mq, each sees another window: in the order of
    their positions, not this one), nor have padding tokens and positions below 0 (ctx_len, q_start, total: as cache_rows)."""
    csa2._need("window_rows", window > 0)
    pos, own = cache_rows(ctx_len, q_start, max_ctx=1 << 31, total=total)
    if ctx_len.numel() == 0:
        return own
    b = torch.searchsorted(q_start.long()[1:].contiguous(), torch.arange(pos.numel(), device=pos.device), right=True)
    b = b.clamp(max=ctx_len.numel() - 1)
    return torch.where((own >= 0) & (pos >= ctx_len[b] - window), b * window + pos % window, torch.full_like(own, -1))


def run_chunk(cb: ChunkBuffers, stream=None):
    """Enqueue the chunk: three library calls in order on one stream, up to four more for `exact` and `keys`.

    With `exact` the dense attention's outputs pass through bf16 on their way into the joined ones: those are rounded
    once more than a decode step's, which joins in fp32 (by 2^-8 of the dense part)."""
    ex, keys = cb.exact, cb.keys
    csa2._need("run_chunk", ex is None or (ex.swa is None) == (ex.swa_rows is None))
    if ex is not None and ex.ring != 0:
        csa2._need("run_chunk", ex.ring > 0 and ex.ring % csa2.PAGE == 0 and (cb.longest or cb.q.shape[0]) + ex.window - 1 <= ex.ring)
    csa2.csa2_rope_apply(cb.rope, cb.q, cb.pos, y=cb.q, offset=csa2.LATENT, stream=stream)
    if ex is not None:
        csa2.csa2_window_append(cb.rope, cb.x, cb.pos, ex.dst_rows, ex.kv, norm_w=cb.norm_w, eps=cb.eps, stream=stream)
        if ex.swa is not None:
            csa2.csa2_window_append(cb.rope, cb.x, cb.pos, ex.swa_rows, ex.swa, norm_w=cb.norm_w, eps=cb.eps, stream=stream)
    if keys is not None:
        csa2.csa2_idx_k_append(keys.rope, keys.kind, keys.x, None if keys.rope is None else cb.pos, cb.dst_rows, keys.idx_k,
                               keys.cache_rows, offset=keys.offset, norm=keys.norm, norm_w=keys.norm_w, norm_b=keys.norm_b,
                               eps=keys.eps, stream=stream)
    csa2.csa2_kv_append(cb.rope, cb.x, cb.pos, cb.dst_rows, cb.kv_codes, cb.kv_scales, cb.kv_rope, norm_w=cb.norm_w,
                        eps=cb.eps, entry=cb.entry, stream=stream)
    csa2.csa2_dense_attn_chunk(cb.dims, cb.batch, cb.q, cb.q_start, cb.kv_codes, cb.kv_scales, cb.kv_rope, cb.page_table,
                               cb.ctx_len, cb.scale, cb.out, cb.lse, cb.ws, window=cb.window, stream=stream)
    if ex is not None:                               # joined in place
        table = cb.page_table if ex.dims is None and ex.page_table is None else ex.page_table
        csa2.csa2_window_attn_chunk(ex.dims or cb.dims, cb.batch, cb.q, cb.q_start, ex.kv, table, cb.ctx_len, cb.scale,
                                    ex.window, cb.out, cb.lse, ex.ws, sinks=ex.sinks, prev_out=cb.out, prev_lse=cb.lse,
                                    stream=stream)
