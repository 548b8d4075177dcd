"""A decode step over the C ABI: owner-filtered append -> partials -> merge.

``ShardedMlaDecoder`` owns the device buffers of one sharded MLA layer held on
this GPU (the pools of shards [shard_begin, shard_end), the partial outputs,
the merged output and the library workspace), all allocated once through
PyTorch.  Each method is a fixed sequence of C-ABI calls; no arithmetic of the
method happens here.

The library's host work per call depends only on shapes, pointers and the
device (every length is read on the device), and nothing here synchronises or
allocates per call, so a whole ``step`` can be captured once in a CUDA graph
(``torch.cuda.graph``) and replayed with new lengths, queries and rows written
in place into the captured tensors.

``cache="q4"`` holds the latent rows in 4 bits (416 bytes a row instead of 1152):
the same calls, on the quantising append and the 4-bit partial.

``BlockTables`` keeps the requests' lengths, their block table and the free
pages on the device and moves them from step to step in one call, which also
lists the new tokens' positions and slots.  Ranks that are given the same lengths
build the same tables, so a group of them exchanges none.

With ``evict=True`` a decoder also accumulates the attention weight of its cached rows
(``weigh``, after a decode) and drops the light ones (``evict``, before the tables
shrink); ``append_normed`` takes latent rows as the projection leaves them.
"""

from __future__ import annotations

import torch

from . import (DCP_LSE_BASE_2, DCP_LSE_BASE_E, DCP_ROPE_PAIRS, Q4_ROW_BYTES, Layout, dcp_block_tables, dcp_evict_select,
               dcp_kv_append, dcp_kv_append_q4, dcp_kv_compact, dcp_kv_compact_q4, dcp_kv_norm_rope_append,
               dcp_kv_norm_rope_append_q4, dcp_key_weights_mark, dcp_lse_merge, dcp_mla_decode_partial,
               dcp_mla_decode_partial_q4, dcp_mla_decode_workspace_size, dcp_mla_decode_workspace_size_q4, dcp_mla_key_weights,
               dcp_mla_key_weights_q4, dcp_mla_key_weights_workspace_size, dcp_mla_key_weights_workspace_size_q4)

_CACHES = {"bf16": (576, torch.bfloat16, dcp_kv_append, dcp_mla_decode_partial, dcp_mla_decode_workspace_size),
           "q4": (Q4_ROW_BYTES, torch.uint8, dcp_kv_append_q4, dcp_mla_decode_partial_q4,
                  dcp_mla_decode_workspace_size_q4)}
_NORMED = {"bf16": dcp_kv_norm_rope_append, "q4": dcp_kv_norm_rope_append_q4}
_WEIGH = {"bf16": (dcp_mla_key_weights, dcp_mla_key_weights_workspace_size),
          "q4": (dcp_mla_key_weights_q4, dcp_mla_key_weights_workspace_size_q4)}
_COMPACT = {"bf16": dcp_kv_compact, "q4": dcp_kv_compact_q4}


class ShardedMlaDecoder:
    def __init__(self, layout: Layout, B: int, q_len: int, H: int, pool_pages: int, max_pages: int,
                 scale: float, lse_base: int = DCP_LSE_BASE_E, out_dtype=torch.bfloat16,
                 part_dtype=torch.float32, shard_begin: int = 0, shard_end: int | None = None,
                 device="cuda", cache: str = "bf16", evict: bool = False):
        if cache not in _CACHES:
            raise ValueError(f"unknown cache format {cache!r} (bf16 or q4)")
        width, dtype, self._append, self._partial, workspace_size = _CACHES[cache]
        self.cache = cache
        self.layout = layout
        self.shard_begin = shard_begin
        self.shard_end = layout.n_shards if shard_end is None else shard_end
        n = self.shard_end - self.shard_begin
        self.B, self.q_len, self.H = B, q_len, H
        self.pool_pages, self.max_pages = pool_pages, max_pages
        self.scale = scale
        self.lse_base = lse_base
        dev = torch.device(device)
        self.arena = torch.zeros(n, pool_pages * layout.page_size, width, dtype=dtype, device=dev)
        self.o_part = torch.empty(n, B, q_len, H, 512, dtype=part_dtype, device=dev)
        self.lse_part = torch.empty(n, B, q_len, H, dtype=torch.float32, device=dev)
        self.o = torch.empty(B, q_len, H, 512, dtype=out_dtype, device=dev)
        self.lse = torch.empty(B, q_len, H, dtype=torch.float32, device=dev)
        self._whole = n == layout.n_shards
        self._merged_part = False   # self.lse is of the held shards alone
        if not self._whole:
            self.lse.fill_(float("nan"))    # until merged, or filled by the caller
        ws = workspace_size(layout, self.shard_begin, self.shard_end, B, q_len, H)
        self._weigh, self._weigh_size = _WEIGH[cache]
        if evict:
            ws = max(ws, self._weigh_size(q_len, H))
        self.workspace = torch.empty(max(ws, 256), dtype=torch.uint8, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        if evict:
            rows = max_pages * layout.page_size
            self.weights = torch.zeros(n, B, rows, dtype=torch.float32, device=dev)
            self.kept = torch.full((n, B, rows), -1, dtype=torch.int32, device=dev)
            # requests' positions below it have a weight, or the mark of none (lower an entry when its request loses
            # tokens from the end, to 0 when its slot gets another request)
            self.weighed = torch.zeros(B, dtype=torch.int64, device=dev)
            self._where = torch.zeros(B, dtype=torch.bool, device=dev)

    def append(self, kv_new, pos, req, block_table, stream=None):
        """Place T new latent rows (kv_new [T, 576] bf16 at positions pos of requests req):
        one owner-filtered append, placement computed in the kernel."""
        if kv_new.shape[0] == 0:
            return
        self._append(self.layout, self.shard_begin, self.shard_end, kv_new, pos, req, block_table,
                     self.max_pages, self.arena, self.pool_pages, self.status, stream)

    def append_normed(self, kv, pos, req, block_table, gamma=None, eps=1e-6, inv_freq=None, rope_style=DCP_ROPE_PAIRS,
                      rope_pos=None, stream=None):
        """append of rows kv [T, 576] that are still a projection's output: latent dims RMS-normed, position dims
        rotated by rope_pos (None: pos; they differ once a request has been shortened)."""
        if kv.shape[0] == 0:
            return
        _NORMED[self.cache](self.layout, self.shard_begin, self.shard_end, kv, pos, req, block_table, self.max_pages,
                            self.arena, self.pool_pages, self.status, gamma=gamma, eps=eps, inv_freq=inv_freq,
                            rope_style=rope_style, rope_pos=rope_pos, stream=stream)

    def weigh(self, q, block_table, seq_lens, decay=1.0, stream=None, lse=None):
        """After a decode of q: what weight every cached row got from it is added to decay times what it had.  A request
        with fewer tokens than q has gets none (DCP_STATUS_BAD_LENGTH).

        lse [B, q_len, H] is the merged one of q over all shards, in the decoder's base; None: self.lse, as decode leaves
        it where all shards are held.  With lse, q may have any number of tokens (a prompt's last ones, say)."""
        if lse is None:
            if self._merged_part:
                raise ValueError(f"self.lse is merged over shards [{self.shard_begin}, {self.shard_end}) of "
                                 f"{self.layout.n_shards} alone; pass lse, the one merged over all of them")
            lse = self.lse
        q_len = q.shape[1]
        fits = q_len <= self.q_len or self._weigh_size(q_len, self.H) <= self.workspace.numel()
        self._weigh(self.layout, self.shard_begin, self.shard_end, q, self.arena, self.pool_pages, block_table,
                    self.max_pages, seq_lens, self.scale, self.lse_base, lse, self.weights, self.status,
                    old_lens=self.weighed, decay=decay, workspace=self.workspace if fits else None, stream=stream)
        with torch.cuda.stream(stream):
            if q_len == 1:
                self.weighed.copy_(seq_lens)
            else:
                torch.ge(seq_lens, q_len, out=self._where)
                torch.minimum(self.weighed, seq_lens, out=self.weighed)
                torch.where(self._where, seq_lens, self.weighed, out=self.weighed)
        return self.weights

    def evict(self, block_table, seq_lens, new_lens, sinks=0, recent=0, stream=None):
        """Every shard keeps its share of new_lens positions of each request: the first `sinks`, the last `recent` and
        the heaviest, moved to the front.  Rows that no weigh has seen stay before those that have a weight (theirs is +inf
        until the next weigh).  The tables, which still hold the old lengths, shrink afterwards
        (BlockTables.update(new_lens)).  Returns kept: the rows that stayed."""
        dcp_key_weights_mark(self.layout, self.shard_begin, self.shard_end, self.weighed, seq_lens, self.weights, stream)
        dcp_evict_select(self.layout, self.shard_begin, self.shard_end, seq_lens, new_lens, sinks, recent, self.weights,
                         self.kept, self.status, stream)
        _COMPACT[self.cache](self.layout, self.shard_begin, self.shard_end, self.kept, new_lens, block_table,
                             self.max_pages, self.arena, self.pool_pages, self.status, weights=self.weights,
                             stream=stream)
        with torch.cuda.stream(stream):  # every row that is left has a weight or the mark; a refused request keeps its length
            torch.lt(new_lens, 0, out=self._where)
            torch.minimum(seq_lens, new_lens, out=self.weighed)
            torch.where(self._where, seq_lens, self.weighed, out=self.weighed)
        return self.kept

    def partial(self, q, block_table, seq_lens, stream=None):
        self._partial(self.layout, self.shard_begin, self.shard_end, q, self.arena,
                      self.pool_pages, block_table, self.max_pages, seq_lens, self.scale,
                      self.lse_base, self.o_part, self.lse_part, self.workspace, self.status,
                      stream)

    def merge(self, stream=None):
        n = self.shard_end - self.shard_begin
        self._merged_part = not self._whole
        dcp_lse_merge(self.o_part.view(n, -1, 512), self.lse_part.view(n, -1), self.lse_base,
                      self.o.view(-1, 512), self.lse.view(-1), stream)

    def decode(self, q, block_table, seq_lens, stream=None):
        """Partials of every held shard, then their merge into self.o / self.lse."""
        self.partial(q, block_table, seq_lens, stream)
        self.merge(stream)
        return self.o, self.lse

    def step(self, q, block_table, seq_lens, kv_new=None, pos=None, req=None, stream=None):
        """One decode step: append this step's tokens (if any), then decode."""
        if kv_new is not None:
            self.append(kv_new, pos, req, block_table, stream)
        return self.decode(q, block_table, seq_lens, stream)

    def status_bits(self) -> int:
        return int(self.status.item())


class BlockTables:
    """Lengths, block table and free pages of B requests, all on the device, for either cache.

    ``update(new_lens)`` moves the requests to their new lengths and fills ``pos``
    and ``req`` (``max_tokens`` entries; -1 behind the last new token) and
    ``cu_tokens``; ``block_table`` and ``seq_lens`` are what the append and the
    partial decode read.  The padded lists go to the append as they are, with as many
    rows (those behind the last token are not read).  With max_tokens 0 no tokens are listed.
    A request of length 0 has o = 0 and lse = -inf in the decode, which flags it BAD_LENGTH."""

    def __init__(self, layout: Layout, B: int, pool_pages: int, max_pages: int, max_tokens: int, device="cuda"):
        dev = torch.device(device)
        self.layout, self.B, self.pool_pages, self.max_pages = layout, B, pool_pages, max_pages
        self.seq_lens = torch.zeros(B, dtype=torch.int64, device=dev)
        self.block_table = torch.full((B, max_pages), -1, dtype=torch.int32, device=dev)
        self.free_pages = torch.arange(pool_pages, dtype=torch.int32, device=dev)
        self.free_state = torch.tensor([0, pool_pages], dtype=torch.int64, device=dev)
        self.cu_tokens = torch.zeros(B + 1, dtype=torch.int64, device=dev)
        self.pos = torch.full((max_tokens,), -1, dtype=torch.int64, device=dev) if max_tokens else None
        self.req = torch.full((max_tokens,), -1, dtype=torch.int32, device=dev) if max_tokens else None
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)

    def update(self, new_lens, stream=None):
        """seq_lens := new_lens (int64 [B] on the device); returns (pos, req) of the new tokens."""
        dcp_block_tables(self.layout, self.seq_lens, new_lens, self.block_table, self.max_pages, self.free_pages,
                         self.free_state, self.cu_tokens, self.status, pos=self.pos, req=self.req, stream=stream)
        return self.pos, self.req

    def status_bits(self) -> int:
        return int(self.status.item())


__all__ = ["ShardedMlaDecoder", "BlockTables", "DCP_LSE_BASE_E", "DCP_LSE_BASE_2"]
