// dcp_cache_q4.cu — writing and reading the 4-bit latent cache (row format:
// dcp_internal.cuh).
//
// Placement (owner, local row, slot) is the slot map's: "PCP / DCP：计算、KV
// 布局与块轮转", section 6; the owner filter is "MLA 的 Decode Context
// Parallelism", section 4, stage 2.
//
// Quantisation of a group of 16 dims with largest magnitude A:
//   s = e4m3(min(A / 7, 448)),  code = clamp(round(x / s), -7, 7)  (0 if s = 0),
// both roundings to nearest, ties to even.  A bf16 x has 8 significant bits and
// s has 4, so x / s is a tie only if it is one exactly, and is otherwise at least
// 2^-9 (relative) away from every tie: correctly rounded fp32 quotients give the
// codes of exact arithmetic.
//
// One warp per token, lane g owns group g (32 bytes in, one 8-byte store of
// codes and one scale byte out), so no value crosses lanes; the 64 rope dims go
// through as 4 bytes a lane.  Memory-bound: 1152 + 416 bytes a token either way.
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

// Checks token (p, b) and returns its place if a held shard owns it; owner -1
// for a padding entry (p = b = -1), a bad one (flagged) or another shard's.
__device__ __forceinline__ Place held_place(int64_t p, int32_t b, const Layout& L, const Table& t, int32_t shard_begin,
                                            int32_t shard_end, int lane, int32_t* status) {
  if (p == -1 && b == -1) return Place{-1, 0};
  if (p < 0 || b < 0 || b >= t.B) {
    if (lane == 0) flag(status, p < 0 ? DCP_STATUS_BAD_POSITION : DCP_STATUS_BAD_REQUEST);
    return Place{-1, 0};
  }
  const Place at = place_of(p, L);
  return at.owner >= shard_begin && at.owner < shard_end ? at : Place{-1, 0};
}

// Pool row of local row `row` of request b, or -1 (flagged).
__device__ __forceinline__ int64_t pool_row(int64_t row, int32_t b, const Layout& L, const Table& t, int lane,
                                            int32_t* status) {
  const int64_t pidx = row < INT32_MAX ? (int32_t)row / (int32_t)L.P : row / L.P;
  if (pidx >= t.max_pages) {
    if (lane == 0) flag(status, DCP_STATUS_BAD_PAGE_INDEX);
    return -1;
  }
  const int64_t page = __ldg(t.bt + (int64_t)b * t.stride + pidx);
  if (page < 0 || page >= t.pool_pages) {
    if (lane == 0) flag(status, DCP_STATUS_BAD_PAGE_ID);
    return -1;
  }
  return page * L.P + (row - pidx * L.P);
}

// 16 bf16 dims -> their two words of codes and the scale byte.
__device__ __forceinline__ uint2 quantise16(const uint4 (&x)[2], uint32_t& scale) {
  float v[16];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&x[j]);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = __bfloat1622float2(h[k]);
      v[8 * j + 2 * k] = f.x;
      v[8 * j + 2 * k + 1] = f.y;
    }
  }
  float top = 0.f;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    top = fmaxf(top, fabsf(v[i]));
    nan |= v[i] != v[i];
  }
  // a NaN makes its whole group one
  scale = nan ? 0x7Fu : (uint32_t)__nv_cvt_float_to_fp8(__fdiv_rn(top, 7.f), __NV_SATFINITE, __NV_E4M3);
  const float s = q4_scales_f32(scale).x;
  uint32_t w[2] = {0x88888888u, 0x88888888u};  // every code 0
  if (s > 0.f) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      w[j] = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float c = fminf(fmaxf(rintf(__fdiv_rn(v[8 * j + i], s)), -7.f), 7.f);
        w[j] |= (uint32_t)((int)c + 8) << (4 * (i >> 1) + 16 * (i & 1));
      }
    }
  }
  return make_uint2(w[0], w[1]);
}

// The source of a moved token's row: row t of kv_new, or the prefill pool's row
// of its position.
struct NewRows {
  const unsigned char* rows;
  __device__ const unsigned char* row(int64_t t, int64_t, int32_t, int, int32_t*) const { return rows + t * (kDk * 2); }
};

struct PoolRows {
  const unsigned char* pool;
  int64_t rows;
  int32_t Ps;
  const int32_t* bt;
  int64_t stride, max_pages;
  __device__ const unsigned char* row(int64_t, int64_t p, int32_t b, int lane, int32_t* status) const {
    const int64_t pidx = p < INT32_MAX ? (int32_t)p / Ps : p / Ps;
    if (pidx >= max_pages) {
      if (lane == 0) flag(status, DCP_STATUS_BAD_PAGE_INDEX);
      return nullptr;
    }
    const int64_t page = __ldg(bt + (int64_t)b * stride + pidx);
    const int64_t r = page * Ps + (p - pidx * Ps);
    if (page < 0 || r >= rows) {
      if (lane == 0) flag(status, DCP_STATUS_BAD_PAGE_ID);
      return nullptr;
    }
    return pool + r * (kDk * 2);
  }
};

template <class Src>
__global__ void __launch_bounds__(256) store_q4_kernel(Layout L, int32_t shard_begin, int32_t shard_end, Src src,
                                                       const int64_t* __restrict__ pos,
                                                       const int32_t* __restrict__ req, int64_t T, Table tab,
                                                       unsigned char* __restrict__ arena, int32_t* status) {
  const int64_t t = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (t >= T) return;
  const int64_t p = __ldg(pos + t);
  const int32_t b = __ldg(req + t);
  const Place at = held_place(p, b, L, tab, shard_begin, shard_end, lane, status);
  if (at.owner < 0) return;
  const unsigned char* from = src.row(t, p, b, lane, status);
  if (!from) return;
  // the row's loads go out before the block-table lookup, so the two latencies overlap
  uint4 x[2];
  x[0] = __ldg(reinterpret_cast<const uint4*>(from) + 2 * lane);
  x[1] = __ldg(reinterpret_cast<const uint4*>(from) + 2 * lane + 1);
  const uint32_t rope = __ldg(reinterpret_cast<const uint32_t*>(from + kDv * 2) + lane);
  const int64_t r = pool_row(at.row, b, L, tab, lane, status);
  if (r < 0) return;
  unsigned char* to = arena + ((at.owner - shard_begin) * tab.pool_pages * L.P + r) * kQ4RowBytes;
  uint32_t scale;
  const uint2 codes = quantise16(x, scale);
  reinterpret_cast<uint2*>(to)[lane] = codes;
  to[kQ4ScaleOff + lane] = (unsigned char)scale;
  reinterpret_cast<uint32_t*>(to + kQ4RopeOff)[lane] = rope;
}

__global__ void __launch_bounds__(256) read_q4_kernel(Layout L, int32_t shard_begin, int32_t shard_end,
                                                      const unsigned char* __restrict__ arena,
                                                      const int64_t* __restrict__ pos,
                                                      const int32_t* __restrict__ req, int64_t T, Table tab,
                                                      unsigned char* __restrict__ kv, int32_t* status) {
  const int64_t t = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (t >= T) return;
  const int64_t p = __ldg(pos + t);
  const int32_t b = __ldg(req + t);
  const Place at = held_place(p, b, L, tab, shard_begin, shard_end, lane, status);
  if (at.owner < 0) return;
  const int64_t r = pool_row(at.row, b, L, tab, lane, status);
  if (r < 0) return;
  const unsigned char* from = arena + ((at.owner - shard_begin) * tab.pool_pages * L.P + r) * kQ4RowBytes;
  const uint2 codes = __ldg(reinterpret_cast<const uint2*>(from) + lane);
  const uint32_t scale = __ldg(from + kQ4ScaleOff + lane);
  const uint32_t rope = __ldg(reinterpret_cast<const uint32_t*>(from + kQ4RopeOff) + lane);
  uint32_t s2[2], off2[2], v[2][4];
  q4_scales(scale, s2, off2);
  q4_values(codes.x, s2[0], off2[0], v[0]);
  q4_values(codes.y, s2[0], off2[0], v[1]);
  unsigned char* to = kv + t * (kDk * 2);
#pragma unroll
  for (int j = 0; j < 2; ++j)
    reinterpret_cast<uint4*>(to)[2 * lane + j] = make_uint4(v[j][0], v[j][1], v[j][2], v[j][3]);
  reinterpret_cast<uint32_t*>(to + kDv * 2)[lane] = rope;
}

constexpr int kThreads = 256;  // 8 tokens per block

int64_t token_blocks(int64_t T) { return (T + kThreads / 32 - 1) / (kThreads / 32); }

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
  const int64_t blocks = token_blocks(T);
  if (blocks > INT32_MAX) return DCP_ERR_UNSUPPORTED;
  store_q4_kernel<<<(unsigned)blocks, kThreads, 0, as_stream(stream)>>>(
      to_layout(layout), shard_begin, shard_end, NewRows{static_cast<const unsigned char*>(kv_new)}, pos, req, T,
      Table{block_table, B, bt_stride, max_pages, pool_pages}, static_cast<unsigned char*>(arena), status);
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
  const int64_t blocks = token_blocks(T);
  if (blocks > INT32_MAX) return DCP_ERR_UNSUPPORTED;
  store_q4_kernel<<<(unsigned)blocks, kThreads, 0, as_stream(stream)>>>(
      to_layout(layout), shard_begin, shard_end,
      PoolRows{static_cast<const unsigned char*>(src_pool), src_pool_rows, src_page_size, src_block_table,
               src_bt_stride, src_max_pages},
      pos, req, T, Table{block_table, B, bt_stride, max_pages, pool_pages}, static_cast<unsigned char*>(arena),
      status);
  return launch_status();
}

extern "C" int32_t dcp_kv_read_q4(const dcp_layout_t* layout, int32_t shard_begin, int32_t shard_end,
                                  const void* arena, int64_t pool_pages, const int64_t* pos, const int32_t* req,
                                  int64_t T, const int32_t* block_table, int32_t B, int64_t bt_stride,
                                  int64_t max_pages, void* kv, int32_t* status, void* stream) {
  if (!cache_args_ok(layout, shard_begin, shard_end, T, B, bt_stride, max_pages, pool_pages)) return DCP_ERR_INVALID;
  if (T == 0) return DCP_OK;
  if (!arena || !pos || !req || !block_table || !kv || misaligned(arena, kv)) return DCP_ERR_INVALID;
  const int64_t blocks = token_blocks(T);
  if (blocks > INT32_MAX) return DCP_ERR_UNSUPPORTED;
  read_q4_kernel<<<(unsigned)blocks, kThreads, 0, as_stream(stream)>>>(
      to_layout(layout), shard_begin, shard_end, static_cast<const unsigned char*>(arena), pos, req, T,
      Table{block_table, B, bt_stride, max_pages, pool_pages}, static_cast<unsigned char*>(kv), status);
  return launch_status();
}
