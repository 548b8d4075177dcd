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
"""

from __future__ import annotations

import torch

from . import (DCP_LSE_BASE_2, DCP_LSE_BASE_E, Q4_ROW_BYTES, Layout, dcp_block_tables, dcp_kv_append,
               dcp_kv_append_q4, dcp_lse_merge, dcp_mla_decode_partial, dcp_mla_decode_partial_q4,
               dcp_mla_decode_workspace_size, dcp_mla_decode_workspace_size_q4)

_CACHES = {"bf16": (576, torch.bfloat16, dcp_kv_append, dcp_mla_decode_partial, dcp_mla_decode_workspace_size),
           "q4": (Q4_ROW_BYTES, torch.uint8, dcp_kv_append_q4, dcp_mla_decode_partial_q4,
                  dcp_mla_decode_workspace_size_q4)}


class ShardedMlaDecoder:
    def __init__(self, layout: Layout, B: int, q_len: int, H: int, pool_pages: int, max_pages: int,
                 scale: float, lse_base: int = DCP_LSE_BASE_E, out_dtype=torch.bfloat16,
                 part_dtype=torch.float32, shard_begin: int = 0, shard_end: int | None = None,
                 device="cuda", cache: str = "bf16"):
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
        ws = workspace_size(layout, self.shard_begin, self.shard_end, B, q_len, H)
        self.workspace = torch.empty(max(ws, 256), dtype=torch.uint8, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)

    def append(self, kv_new, pos, req, block_table, stream=None):
        """Place T new latent rows (kv_new [T, 576] bf16 at positions pos of requests req):
        one owner-filtered append, placement computed in the kernel."""
        if kv_new.shape[0] == 0:
            return
        self._append(self.layout, self.shard_begin, self.shard_end, kv_new, pos, req, block_table,
                     self.max_pages, self.arena, self.pool_pages, self.status, stream)

    def partial(self, q, block_table, seq_lens, stream=None):
        self._partial(self.layout, self.shard_begin, self.shard_end, q, self.arena,
                      self.pool_pages, block_table, self.max_pages, seq_lens, self.scale,
                      self.lse_base, self.o_part, self.lse_part, self.workspace, self.status,
                      stream)

    def merge(self, stream=None):
        n = self.shard_end - self.shard_begin
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
