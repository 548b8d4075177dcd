// dcp_cache_q4.cu — writing and reading the 4-bit latent cache (row format:
// dcp_internal.cuh).
//
// Placement (owner, local row, slot) is the slot map's: "PCP / DCP：计算、KV
// 布局与块轮转", section 6; the owner filter is "MLA 的 Decode Context
// Parallelism", section 4, stage 2.
//
// Quantisation of a group of 16 dims with largest magnitude A:
//   s = e4m3(min(A / 7, 448)),  code = clamp(round(x / s), -7, 7)  (0 if s = 0),
// both roundings to nearest, ties to even.  The codes are those of exact arithmetic
// without a division per value: a bf16 x has 8 significant bits and s has 4, so
// x / s is a tie n + 1/2 exactly or at least 2^-9 away from every tie, while
// y = x * (1 / s) in fp32 is within 2^-19 of x / s (|x / s| < 8).  Rounding y to a
// multiple of 2^-12 therefore restores a tie and makes none.  (With 16 fp32
// divisions a lane the kernel was bound by them: 18 us for 32768 rows.)
//
// A warp serves `per_warp` tokens: a lane each looks up their places, so that
// positions, requests and block-table entries are one latency for all of them;
// then lane g takes group g of each token (32 bytes in, 8 bytes of codes and a
// scale byte out, or the other way), four tokens' loads ahead of their stores, and
// no value crosses lanes; the 64 rope dims go through as 4 bytes a lane.
// Memory-bound for long lists: 1152 + 416 bytes a token either way.
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

// Pool row (over all held pools) of token (p, b), or -1 for a padding entry
// (p = b = -1), another shard's token, or a bad one (flagged).
__device__ __forceinline__ int64_t held_row(int64_t p, int32_t b, const Layout& L, const Table& t, int32_t shard_begin,
                                            int32_t shard_end, int32_t* status) {
  if (p == -1 && b == -1) return -1;
  if (p < 0 || b < 0 || b >= t.B) {
    flag(status, p < 0 ? DCP_STATUS_BAD_POSITION : DCP_STATUS_BAD_REQUEST);
    return -1;
  }
  const Place at = place_of(p, L);
  if (at.owner < shard_begin || at.owner >= shard_end) return -1;
  const int64_t pidx = at.row < INT32_MAX ? (int32_t)at.row / (int32_t)L.P : at.row / L.P;
  if (pidx >= t.max_pages) {
    flag(status, DCP_STATUS_BAD_PAGE_INDEX);
    return -1;
  }
  const int64_t page = __ldg(t.bt + (int64_t)b * t.stride + pidx);
  if (page < 0 || page >= t.pool_pages) {
    flag(status, DCP_STATUS_BAD_PAGE_ID);
    return -1;
  }
  return ((at.owner - shard_begin) * t.pool_pages + page) * L.P + (at.row - pidx * L.P);
}

// 16 bf16 dims -> their two words of codes and the scale byte.
__device__ __forceinline__ uint2 quantise16(const uint4 (&x)[2], uint32_t& scale) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(x);
  __nv_bfloat162 top2 = __habs2(h[0]);
#pragma unroll
  for (int k = 1; k < 8; ++k) top2 = __hmax2_nan(top2, __habs2(h[k]));
  // a NaN makes its whole group one (and e4m3's only NaN, 0x7f, its scale)
  const float top = __bfloat162float(__hmax_nan(top2.x, top2.y));
  scale = (uint32_t)__nv_cvt_float_to_fp8(__fdiv_rn(top, 7.f), __NV_SATFINITE, __NV_E4M3);
  const float s = q4_scales_f32(scale).x;
  if (!(s > 0.f)) return make_uint2(0x88888888u, 0x88888888u);  // every code 0
  const float inv = __frcp_rn(s);
  constexpr float kSnap = 1.5f * 2048.f;               // + and - this: to a multiple of 2^-12
  constexpr float kInt = 1.5f * 8388608.f + 8.f;       // + this: code + 8 in the low mantissa bits
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float2 f = __bfloat1622float2(h[k]);
    const float a = fminf(fmaxf(f.x * inv, -7.f), 7.f), b = fminf(fmaxf(f.y * inv, -7.f), 7.f);
    const uint32_t na = __float_as_uint(__fadd_rn(__fsub_rn(__fadd_rn(a, kSnap), kSnap), kInt)) & 15u;
    const uint32_t nb = __float_as_uint(__fadd_rn(__fsub_rn(__fadd_rn(b, kSnap), kSnap), kInt)) & 15u;
    w[k >> 2] |= (na | nb << 16) << (4 * (k & 3));
  }
  return make_uint2(w[0], w[1]);
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

constexpr int kAhead = 4;  // tokens whose loads are in flight before their stores

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
  if (lane < n) {
    const int64_t p = __ldg(pos + t0 + lane);
    const int32_t b = __ldg(req + t0 + lane);
    to = held_row(p, b, L, tab, shard_begin, shard_end, status);
    if (to >= 0) from = src.row(t0 + lane, p, b, status);
  }
  for (int i = 0; i < n; i += kAhead) {
    uint4 x[kAhead][2];
    uint32_t rope[kAhead];
    int64_t f[kAhead];
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
      f[e] = __shfl_sync(0xffffffffu, from, i + e);
      if (i + e >= n) f[e] = -1;
      if (f[e] < 0) continue;
      const unsigned char* row = src.base + f[e] * (kDk * 2);
      x[e][0] = __ldg(reinterpret_cast<const uint4*>(row) + 2 * lane);
      x[e][1] = __ldg(reinterpret_cast<const uint4*>(row) + 2 * lane + 1);
      rope[e] = __ldg(reinterpret_cast<const uint32_t*>(row + kDv * 2) + lane);
    }
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
      const int64_t r = __shfl_sync(0xffffffffu, to, i + e);
      if (f[e] < 0) continue;
      unsigned char* row = arena + r * kQ4RowBytes;
      uint32_t scale;
      const uint2 codes = quantise16(x[e], scale);
      reinterpret_cast<uint2*>(row)[lane] = codes;
      row[kQ4ScaleOff + lane] = (unsigned char)scale;
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
  if (lane < n) from = held_row(__ldg(pos + t0 + lane), __ldg(req + t0 + lane), L, tab, shard_begin, shard_end, status);
  for (int i = 0; i < n; i += kAhead) {
    uint2 codes[kAhead];
    uint32_t scale[kAhead], rope[kAhead];
    int64_t f[kAhead];
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
      f[e] = __shfl_sync(0xffffffffu, from, i + e);
      if (i + e >= n) f[e] = -1;
      if (f[e] < 0) continue;
      const unsigned char* row = arena + f[e] * kQ4RowBytes;
      codes[e] = __ldg(reinterpret_cast<const uint2*>(row) + lane);
      scale[e] = __ldg(row + kQ4ScaleOff + lane);
      rope[e] = __ldg(reinterpret_cast<const uint32_t*>(row + kQ4RopeOff) + lane);
    }
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
      if (f[e] < 0) continue;
      uint32_t s2[2], off2[2], v[2][4];
      q4_scales(scale[e], s2, off2);
      q4_values(codes[e].x, s2[0], off2[0], v[0]);
      q4_values(codes[e].y, s2[0], off2[0], v[1]);
      unsigned char* row = kv + (t0 + i + e) * (kDk * 2);
#pragma unroll
      for (int j = 0; j < 2; ++j)
        reinterpret_cast<uint4*>(row)[2 * lane + j] = make_uint4(v[j][0], v[j][1], v[j][2], v[j][3]);
      reinterpret_cast<uint32_t*>(row + kDv * 2)[lane] = rope[e];
    }
  }
}

constexpr int kThreads = 256;  // 8 warps

// Tokens a warp serves: one while the list does not fill the card (4864 warps are
// 32 on each of 152 SMs), then as many as keep that many warps, up to 32.
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
