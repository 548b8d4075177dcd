// dcp_rows.cuh — what the kernels that write or read cache rows share: where a token
// goes, and how a token list is spread over warps.
#pragma once

#include "dcp_internal.cuh"

using namespace dcp;

namespace {

struct Place {
  int64_t owner, row;
};

// Owner and local row of position p (32-bit arithmetic below 2^31).
__device__ __forceinline__ Place place_of(int64_t p, const Layout& L) {
  if (p < INT32_MAX) {
    const int32_t p32 = (int32_t)p, I = (int32_t)L.I, N = (int32_t)L.N, blk = p32 / I;
    return Place{blk % N, (int64_t)(blk / N) * I + p32 % I};
  }
  return Place{owner_of(p, L), local_row_of(p, L)};
}

struct Table {
  const int32_t* bt;
  int32_t B;
  int64_t stride, max_pages, pool_pages;
};

// Where a token goes: its block-table entry is loaded, but not looked at yet, so
// that the loads of its row can go out in the same latency.
struct Spot {
  int64_t page;  // block-table entry
  int64_t pool;  // first row of its shard's pool, -1: nothing to do
  int64_t in_page;
};

// The spot of token (p, b); none for a padding entry (p = b = -1), another shard's
// token, or a bad one (flagged).
__device__ __forceinline__ Spot find_spot(int64_t p, int32_t b, const Layout& L, const Table& t, int32_t shard_begin,
                                          int32_t shard_end, int32_t* status) {
  if (is_padding(p, b)) return Spot{-1, -1, 0};
  if (p < 0 || b < 0 || b >= t.B) {
    flag(status, p < 0 ? DCP_STATUS_BAD_POSITION : DCP_STATUS_BAD_REQUEST);
    return Spot{-1, -1, 0};
  }
  const Place at = place_of(p, L);
  if (at.owner < shard_begin || at.owner >= shard_end) return Spot{-1, -1, 0};
  const int64_t pidx = at.row < INT32_MAX ? (int32_t)at.row / (int32_t)L.P : at.row / L.P;
  if (pidx >= t.max_pages) {
    flag(status, DCP_STATUS_BAD_PAGE_INDEX);
    return Spot{-1, -1, 0};
  }
  return Spot{__ldg(t.bt + (int64_t)b * t.stride + pidx), (at.owner - shard_begin) * t.pool_pages * L.P,
              at.row - pidx * L.P};
}

// Its row over all held pools, or -1 (a bad page is flagged).
__device__ __forceinline__ int64_t row_of(const Spot& s, const Layout& L, const Table& t, int32_t* status) {
  if (s.pool < 0) return -1;
  if (s.page < 0 || s.page >= t.pool_pages) {
    flag(status, DCP_STATUS_BAD_PAGE_ID);
    return -1;
  }
  return s.pool + s.page * L.P + s.in_page;
}

constexpr int kThreads = 256;  // 8 warps

// Tokens a warp serves: one while the list does not fill the card (4864 warps are
// 32 on each of 152 SMs), then as many as keep that many warps, up to 32.  Writing
// 3708 rows takes 4.7 us with 1, 5.6 with 8 and 14.8 with 32; 32768 rows 22.2, 11.7
// and 14.9; 262144 rows 183, 73 and 70.
int tokens_per_warp(int64_t T) {
  int n = 1;
  while (n < 32 && T > 4864 * (int64_t)n) n *= 2;
  return n;
}

int64_t token_blocks(int64_t T, int per_warp) {
  const int64_t per_block = (int64_t)(kThreads / 32) * per_warp;
  return (T + per_block - 1) / per_block;
}

bool misaligned(const void* a, const void* b) {
  return ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b)) & 15) != 0;
}

bool cache_args_ok(const dcp_layout_t* layout, int32_t shard_begin, int32_t shard_end, int64_t T, int32_t B,
                   int64_t bt_stride, int64_t max_pages, int64_t pool_pages) {
  return layout_ok(layout) && shard_begin >= 0 && shard_end <= layout->n_shards && shard_begin < shard_end && T >= 0 &&
         B >= 1 && max_pages >= 1 && bt_stride >= max_pages && pool_pages >= 1;
}

}  // namespace
