// dcp_cache_q4.cu — writing and reading the 4-bit latent cache (row format:
// dcp_internal.cuh).
//
// Placement (owner, local row, slot) is the slot map's: "PCP / DCP：计算、KV
// 布局与块轮转", section 6; the owner filter is "MLA 的 Decode Context
// Parallelism", section 4, stage 2.
//
// Quantisation of a group of 16 dims with largest magnitude A:
//   s = e4m3(min(A / 7, 448)),  code = clamp(round(x / s), -7, 7)  (0 if s = 0),
// both roundings to nearest, ties to even.  Both are those of exact arithmetic,
// without a division: a bf16 x has 8 significant bits and s has 4, so x / s is a tie
// n + 1/2 exactly or at least 2^-9 away from every tie, while x * (1 / s) in fp32 is
// within 2^-19 of x / s (|x / s| < 8).  Rounding it to a multiple of 2^-11 therefore
// restores a tie and makes none.  A / 7 likewise: rounded to 12 significant bits, it
// lies on a midpoint of two e4m3 values only if it does exactly (those have 5).
// (With 17 fp32 divisions a lane the kernel was bound by them: 122 us for 262143
// rows, against 72 now.)
//
// A warp serves `per_warp` tokens: a lane each looks up their places, so that
// positions, requests and block-table entries are one latency for all of them; then
// the whole warp takes a token at a time, several tokens' loads ahead of their stores.
// Lane l has dims [8 l, 8 l + 8) and [256 + 8 l, 256 + 8 l + 8), one word of codes
// each, so that every access is one run of the row: 512 bytes of bf16, 128 of codes.
// A group is two neighbouring lanes' (one shuffle for its magnitude); the 64 rope
// dims go through as 4 bytes a lane.  Memory-bound for long lists: 1152 + 416 bytes a
// token either way; 262143 rows in 72 us written (5.7 TB/s) and 76 us read (5.4 TB/s).
// A list of a few rows is two or three memory latencies, 2.7 us in a captured graph.
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

// The source row of a moved token, or -1: row t of kv_new, or the prefill pool's
// row of its position.
struct NewRows {
  const unsigned char* base;
  __device__ int64_t row(int64_t t, int64_t, int32_t, int32_t*) const { return t; }
};

struct PoolRows {
  const unsigned char* base;
  int64_t rows;
  int32_t Ps;
  const int32_t* bt;
  int64_t stride, max_pages;
  __device__ int64_t row(int64_t, int64_t p, int32_t b, int32_t* status) const {
    const int64_t pidx = p < INT32_MAX ? (int32_t)p / Ps : p / Ps;
    if (pidx >= max_pages) {
      flag(status, DCP_STATUS_BAD_PAGE_INDEX);
      return -1;
    }
    const int64_t page = __ldg(bt + (int64_t)b * stride + pidx);
    const int64_t r = page * Ps + (p - pidx * Ps);
    if (page < 0 || r >= rows) {
      flag(status, DCP_STATUS_BAD_PAGE_ID);
      return -1;
    }
    return r;
  }
};

// Tokens whose loads are in flight before their stores.  262143 rows: writing takes
// 72 us with 4 and 91 with 8 (fewer warps fit), reading 88 and 76.
constexpr int kStoreAhead = 4, kReadAhead = 8;

template <class Src>
__global__ void __launch_bounds__(256) store_q4_kernel(Layout L, int32_t shard_begin, int32_t shard_end, Src src,
                                                       const int64_t* __restrict__ pos,
                                                       const int32_t* __restrict__ req, int64_t T, int per_warp,
                                                       Table tab, unsigned char* __restrict__ arena,
                                                       int32_t* status) {
  const int64_t t0 = (blockIdx.x * (int64_t)(blockDim.x / 32) + (threadIdx.x >> 5)) * per_warp;
  const int lane = threadIdx.x & 31;
  const int n = (int)min((int64_t)per_warp, T - t0);  // not above 0: no token
  int64_t from = -1, to = -1;                         // lane: source and pool row of token t0 + lane
  Spot spot{-1, -1, 0};
  if (lane < n) {
    const int64_t p = __ldg(pos + t0 + lane);
    const int32_t b = __ldg(req + t0 + lane);
    spot = find_spot(p, b, L, tab, shard_begin, shard_end, status);
    if (spot.pool >= 0) from = src.row(t0 + lane, p, b, status);
  }
  for (int i = 0; i < n; i += kStoreAhead) {
    uint4 x[kStoreAhead][2];
    uint32_t rope[kStoreAhead];
    int64_t f[kStoreAhead];
#pragma unroll
    for (int e = 0; e < kStoreAhead; ++e) {
      f[e] = __shfl_sync(0xffffffffu, from, i + e);
      if (i + e >= n) f[e] = -1;
      x[e][0] = x[e][1] = make_uint4(0, 0, 0, 0);
      if (f[e] < 0) continue;
      const unsigned char* row = src.base + f[e] * (kDk * 2);
      x[e][0] = __ldg(reinterpret_cast<const uint4*>(row) + lane);
      x[e][1] = __ldg(reinterpret_cast<const uint4*>(row) + 32 + lane);
      rope[e] = __ldg(reinterpret_cast<const uint32_t*>(row + kDv * 2) + lane);
    }
    if (i == 0 && from >= 0) to = row_of(spot, L, tab, status);
#pragma unroll
    for (int e = 0; e < kStoreAhead; ++e) {
      const int64_t r = __shfl_sync(0xffffffffu, to, i + e);
      // largest magnitudes of this lane's two groups: its own 8 dims and its neighbour's
      const __nv_bfloat162 mine = __nv_bfloat162(top8(x[e][0]), top8(x[e][1]));
      const __nv_bfloat162 top2 = __hmax2_nan(mine, __shfl_xor_sync(0xffffffffu, mine, 1));
      if (f[e] < 0 || r < 0) continue;
      unsigned char* row = arena + r * kQ4RowBytes;
      const float2 top = __bfloat1622float2(top2);
      const uint32_t scales = __nv_cvt_float2_to_fp8x2(make_float2(seventh(top.x), seventh(top.y)), __NV_SATFINITE,
                                                       __NV_E4M3);
      const float2 s = q4_scales_f32(scales);
      reinterpret_cast<uint32_t*>(row)[lane] = codes8(x[e][0], s.x, top.x);
      reinterpret_cast<uint32_t*>(row)[32 + lane] = codes8(x[e][1], s.y, top.y);
      // an even lane writes the scale of group l / 2, its neighbour that of group 16 + l / 2
      row[kQ4ScaleOff + 16 * (lane & 1) + (lane >> 1)] = (unsigned char)(lane & 1 ? scales >> 8 : scales);
      reinterpret_cast<uint32_t*>(row + kQ4RopeOff)[lane] = rope[e];
    }
  }
}

__global__ void __launch_bounds__(256) read_q4_kernel(Layout L, int32_t shard_begin, int32_t shard_end,
                                                      const unsigned char* __restrict__ arena,
                                                      const int64_t* __restrict__ pos,
                                                      const int32_t* __restrict__ req, int64_t T, int per_warp,
                                                      Table tab, unsigned char* __restrict__ kv, int32_t* status) {
  const int64_t t0 = (blockIdx.x * (int64_t)(blockDim.x / 32) + (threadIdx.x >> 5)) * per_warp;
  const int lane = threadIdx.x & 31;
  const int n = (int)min((int64_t)per_warp, T - t0);
  int64_t from = -1;  // lane: pool row of token t0 + lane
  if (lane < n)
    from = row_of(find_spot(__ldg(pos + t0 + lane), __ldg(req + t0 + lane), L, tab, shard_begin, shard_end, status), L,
                  tab, status);
  for (int i = 0; i < n; i += kReadAhead) {
    uint32_t codes[kReadAhead][2], scales[kReadAhead], rope[kReadAhead];
    int64_t f[kReadAhead];
#pragma unroll
    for (int e = 0; e < kReadAhead; ++e) {
      f[e] = __shfl_sync(0xffffffffu, from, i + e);
      if (i + e >= n) f[e] = -1;
      if (f[e] < 0) continue;
      const unsigned char* row = arena + f[e] * kQ4RowBytes;
      codes[e][0] = __ldg(reinterpret_cast<const uint32_t*>(row) + lane);
      codes[e][1] = __ldg(reinterpret_cast<const uint32_t*>(row) + 32 + lane);
      scales[e] = __ldg(row + kQ4ScaleOff + (lane >> 1)) | (uint32_t)__ldg(row + kQ4ScaleOff + 16 + (lane >> 1)) << 8;
      rope[e] = __ldg(reinterpret_cast<const uint32_t*>(row + kQ4RopeOff) + lane);
    }
#pragma unroll
    for (int e = 0; e < kReadAhead; ++e) {
      if (f[e] < 0) continue;
      uint32_t s2[2], off2[2];
      q4_scales(scales[e], s2, off2);
      unsigned char* row = kv + (t0 + i + e) * (kDk * 2);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t v[4];
        q4_values(codes[e][j], s2[j], off2[j], v);
        reinterpret_cast<uint4*>(row)[32 * j + lane] = make_uint4(v[0], v[1], v[2], v[3]);
      }
      reinterpret_cast<uint32_t*>(row + kDv * 2)[lane] = rope[e];
    }
  }
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

extern "C" int32_t dcp_kv_append_q4(const dcp_layout_t* layout, int32_t shard_begin, int32_t shard_end,
                                    const void* kv_new, const int64_t* pos, const int32_t* req, int64_t T,
                                    const int32_t* block_table, int32_t B, int64_t bt_stride, int64_t max_pages,
                                    void* arena, int64_t pool_pages, int32_t* status, void* stream) {
  if (!cache_args_ok(layout, shard_begin, shard_end, T, B, bt_stride, max_pages, pool_pages)) return DCP_ERR_INVALID;
  if (T == 0) return DCP_OK;
  if (!kv_new || !pos || !req || !block_table || !arena || misaligned(kv_new, arena)) return DCP_ERR_INVALID;
  const int per_warp = tokens_per_warp(T);
  const int64_t blocks = token_blocks(T, per_warp);
  if (blocks > INT32_MAX) return DCP_ERR_UNSUPPORTED;
  store_q4_kernel<<<(unsigned)blocks, kThreads, 0, as_stream(stream)>>>(
      to_layout(layout), shard_begin, shard_end, NewRows{static_cast<const unsigned char*>(kv_new)}, pos, req, T,
      per_warp, Table{block_table, B, bt_stride, max_pages, pool_pages}, static_cast<unsigned char*>(arena), status);
  return launch_status();
}

extern "C" int32_t dcp_kv_relayout_q4(const dcp_layout_t* layout, int32_t shard_begin, int32_t shard_end,
                                      const void* src_pool, int64_t src_pool_rows, int32_t src_page_size,
                                      const int32_t* src_block_table, int64_t src_bt_stride, int64_t src_max_pages,
                                      const int64_t* pos, const int32_t* req, int64_t T, int32_t B,
                                      const int32_t* block_table, int64_t bt_stride, int64_t max_pages, void* arena,
                                      int64_t pool_pages, int32_t* status, void* stream) {
  if (!cache_args_ok(layout, shard_begin, shard_end, T, B, bt_stride, max_pages, pool_pages) || src_page_size < 1 ||
      src_pool_rows < 1 || src_max_pages < 1 || src_bt_stride < src_max_pages)
    return DCP_ERR_INVALID;
  if (T == 0) return DCP_OK;
  if (!src_pool || !src_block_table || !pos || !req || !block_table || !arena || !status ||
      misaligned(src_pool, arena))
    return DCP_ERR_INVALID;
  const int per_warp = tokens_per_warp(T);
  const int64_t blocks = token_blocks(T, per_warp);
  if (blocks > INT32_MAX) return DCP_ERR_UNSUPPORTED;
  store_q4_kernel<<<(unsigned)blocks, kThreads, 0, as_stream(stream)>>>(
      to_layout(layout), shard_begin, shard_end,
      PoolRows{static_cast<const unsigned char*>(src_pool), src_pool_rows, src_page_size, src_block_table,
               src_bt_stride, src_max_pages},
      pos, req, T, per_warp, Table{block_table, B, bt_stride, max_pages, pool_pages},
      static_cast<unsigned char*>(arena), status);
  return launch_status();
}

extern "C" int32_t dcp_kv_read_q4(const dcp_layout_t* layout, int32_t shard_begin, int32_t shard_end,
                                  const void* arena, int64_t pool_pages, const int64_t* pos, const int32_t* req,
                                  int64_t T, const int32_t* block_table, int32_t B, int64_t bt_stride,
                                  int64_t max_pages, void* kv, int32_t* status, void* stream) {
  if (!cache_args_ok(layout, shard_begin, shard_end, T, B, bt_stride, max_pages, pool_pages)) return DCP_ERR_INVALID;
  if (T == 0) return DCP_OK;
  if (!arena || !pos || !req || !block_table || !kv || misaligned(arena, kv)) return DCP_ERR_INVALID;
  const int per_warp = tokens_per_warp(T);
  const int64_t blocks = token_blocks(T, per_warp);
  if (blocks > INT32_MAX) return DCP_ERR_UNSUPPORTED;
  read_q4_kernel<<<(unsigned)blocks, kThreads, 0, as_stream(stream)>>>(
      to_layout(layout), shard_begin, shard_end, static_cast<const unsigned char*>(arena), pos, req, T, per_warp,
      Table{block_table, B, bt_stride, max_pages, pool_pages}, static_cast<unsigned char*>(kv), status);
  return launch_status();
}
