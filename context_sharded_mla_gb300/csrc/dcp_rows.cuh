// dcp_rows.cuh — what the kernels that write or read cache rows share: where a token
// goes, the 4-bit codes of its values (row format and quantiser: dcp_internal.cuh and
// dcp_cache_q4.cu), and how a token list is spread over warps.
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

// Largest magnitude of 8 bf16 values; a NaN among them gives NaN.
__device__ __forceinline__ __nv_bfloat16 top8(const uint4& x) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&x);
  const __nv_bfloat162 a = __hmax2_nan(__habs2(h[0]), __habs2(h[1])), b = __hmax2_nan(__habs2(h[2]), __habs2(h[3]));
  const __nv_bfloat162 c = __hmax2_nan(a, b);
  return __hmax_nan(c.x, c.y);
}

// A / 7 to 12 significant bits (an infinity stays one; a NaN's bits could wrap).
__device__ __forceinline__ float seventh(float top) {
  const float q = __uint_as_float((__float_as_uint(top * (1.f / 7.f)) + 0x800u) & 0xFFFFF000u);
  return top != top ? top : q;
}

__device__ __forceinline__ float reciprocal(float s) {  // within 1 ulp
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return r;
}

// Quotients from here on are clamped before they are rounded.  x / s is at most 7.46875 or
// at least 7.5 (8 significant bits over 4), so the limit is one between the two that a
// reciprocal one ulp off cannot cross.  (7.5 itself is crossed: it would become code 8, in
// the next dim's bits.)
constexpr float kClampFrom = 7.499f;

// The word of codes of 8 bf16 values under scale s, whose group's largest magnitude is
// `top`.  A sum with kSnap ends at a multiple of 2^-11, one with kInt at a whole number
// that its low mantissa bits hold as code + 8.
__device__ __forceinline__ uint32_t codes8(const uint4& x, float s, float top) {
  constexpr float kSnap = 1.5f * 4096.f, kInt = 1.5f * 8388608.f + 8.f;
  if (!(s > 0.f)) return 0x88888888u;  // scale 0 or NaN: every code 0
  const float inv = reciprocal(s);
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&x);
  // only a scale that was clamped, or is one of the few smallest, leaves |x / s| above 7.5
  const bool clamp = !(top * inv < kClampFrom);
  uint32_t w = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float2 f = __bfloat1622float2(h[k]);
    if (clamp) {
      f.x = fminf(fmaxf(f.x, -7.f * s), 7.f * s);
      f.y = fminf(fmaxf(f.y, -7.f * s), 7.f * s);
    }
    const uint32_t a = __float_as_uint(__fadd_rn(__fmaf_rn(f.x, inv, kSnap), kInt - kSnap));
    const uint32_t b = __float_as_uint(__fadd_rn(__fmaf_rn(f.y, inv, kSnap), kInt - kSnap));
    w |= __byte_perm(a, b, 0x5410) << (4 * k);
  }
  return w;
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
