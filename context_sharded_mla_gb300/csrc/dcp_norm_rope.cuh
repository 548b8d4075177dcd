// dcp_norm_rope.cuh — RMS norm and rotation of a row, and the append that does both on its
// way into a pool (dcp_norm_rope.cu: the mathematics, and the bf16 cache; dcp_cache_q4.cu:
// the 4-bit one).
#pragma once

#include "dcp_rows.cuh"

namespace {

constexpr int kRope = kDk - kDv;  // position dims

// A frequency (radians a position) as a step of 2^-64 turns, modulo one turn.
__device__ __forceinline__ uint64_t turn_step(float inv_freq) {
  const double turns = (double)inv_freq * 0.15915494309189535;  // 1 / 2 pi
  return __double2ull_rn((turns - floor(turns)) * 18446744073709551616.0);
}

struct Turn {
  float s, c;
};

__device__ __forceinline__ Turn turn_of(uint64_t step, int64_t pos) {
  const uint64_t f = step * (uint64_t)pos;  // modulo a turn
  Turn t;
  sincospif((float)(int32_t)(f >> 32) * 0x1p-31f, &t.s, &t.c);  // half turns in [-1, 1], rounded once: 2^-23 rad
  return t;
}

__device__ __forceinline__ void unpack8(const uint4& u, float (&v)[8]) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = __bfloat1622float2(h[k]);
    v[2 * k] = f.x;
    v[2 * k + 1] = f.y;
  }
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  uint4 u;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
  for (int k = 0; k < 4; ++k) h[k] = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
  return u;
}

// The frequencies' steps into shared memory (f64 runs at 2 operations a clock and SM: once a block, not once a warp).
__device__ __forceinline__ void load_steps(const float* inv_freq, uint64_t* steps) {
  if (inv_freq && threadIdx.x < kRope / 2) steps[threadIdx.x] = turn_step(__ldg(inv_freq + threadIdx.x));
}

// 8 normed values: x * inv * gamma.
__device__ __forceinline__ void scale8(float (&v)[8], float inv, const float (&g)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = v[k] * inv * g[k];
}

__device__ __forceinline__ float square8(const float (&v)[8], float sum) {
#pragma unroll
  for (int k = 0; k < 8; ++k) sum = fmaf(v[k], v[k], sum);
  return sum;
}

// ---------------------------------------------------------------- latent rows
struct RowArgs {
  const unsigned char* kv;  // bf16 rows, `stride` bytes apart
  int64_t stride;
  const void* gamma;
  int gamma_bf16;
  float eps;
  const float* inv_freq;
  int halves;
  const int64_t* rope_pos;
};

// Tokens whose loads are in flight before their stores, 32768 tokens in a captured graph: 14.4 us with 2 and four blocks
// an SM (4-bit 20); when that took 14.9 it was 16.1 with 4 and two blocks, 18.4 with 3 and three, 16.0 with 1 and five.
// Eight rows a warp copied asynchronously into shared memory: 16.6.
constexpr int kRowAhead = 2;

// A bf16 row's first 512 dims: lane l has dims [8 l, 8 l + 8) and [256 + 8 l, 256 + 8 l + 8).
struct Bf16Row {
  static constexpr int kBytes = kDk * 2, kRopeAt = kDv * 2;
  uint4 x0, x1;
  __device__ explicit Bf16Row(const uint4 (&x)[2]) : x0(x[0]), x1(x[1]) {}
  __device__ void store(unsigned char* row, int lane) const {
    reinterpret_cast<uint4*>(row)[lane] = x0;
    reinterpret_cast<uint4*>(row)[32 + lane] = x1;
  }
};

template <class Row>
__global__ void __launch_bounds__(256, 4) norm_rope_store_kernel(Layout L, int32_t shard_begin, int32_t shard_end,
                                                              RowArgs in, const int64_t* __restrict__ pos,
                                                              const int32_t* __restrict__ req, int64_t T, int per_warp,
                                                              Table tab, unsigned char* __restrict__ arena,
                                                              int32_t* status) {
  __shared__ __align__(16) float gamma_s[kDv];
  __shared__ uint64_t steps_s[kRope / 2];
  const int64_t t0 = (blockIdx.x * (int64_t)(blockDim.x / 32) + (threadIdx.x >> 5)) * per_warp;
  const int lane = threadIdx.x & 31;
  const int n = (int)min((int64_t)per_warp, T - t0);
  // norm weights in f32, as four planes: [2 j + h][lane] holds dims 256 j + 8 lane + 4 h + [0, 4)
  if (in.gamma)
    for (int i = threadIdx.x; i < kDv; i += blockDim.x)
      gamma_s[128 * (2 * (i >> 8) + (i >> 2 & 1)) + 4 * (i >> 3 & 31) + (i & 3)] =
          in.gamma_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(in.gamma)[i])
                        : static_cast<const float*>(in.gamma)[i];
  load_steps(in.inv_freq, steps_s);
  __syncthreads();
  if (n <= 0) return;
  Spot spot{-1, -1, 0};
  int64_t angle_pos = 0, to = -1;  // lane: of token t0 + lane
  if (lane < n) {
    const int64_t p = __ldg(pos + t0 + lane);
    angle_pos = in.rope_pos ? __ldg(in.rope_pos + t0 + lane) : p;
    spot = find_spot(p, __ldg(req + t0 + lane), L, tab, shard_begin, shard_end, status);
  }
  const uint64_t step = in.inv_freq ? steps_s[lane] : 0;  // lane: pair `lane`
  for (int i = 0; i < n; i += kRowAhead) {
    uint4 x[kRowAhead][2];
    uint32_t rope[kRowAhead];  // this lane's pair: dims 2 l, 2 l + 1 or l, l + 32
    bool live[kRowAhead];
#pragma unroll
    for (int e = 0; e < kRowAhead; ++e) {
      live[e] = __shfl_sync(0xffffffffu, spot.pool, i + e) >= 0 && i + e < n;
      x[e][0] = x[e][1] = make_uint4(0, 0, 0, 0);
      rope[e] = 0;
      if (!live[e]) continue;
      const unsigned char* row = in.kv + (t0 + i + e) * in.stride;
      x[e][0] = __ldg(reinterpret_cast<const uint4*>(row) + lane);
      x[e][1] = __ldg(reinterpret_cast<const uint4*>(row) + 32 + lane);
      if (in.halves) {
        const unsigned short* r = reinterpret_cast<const unsigned short*>(row + kDv * 2);
        rope[e] = __ldg(r + lane) | (uint32_t)__ldg(r + kRope / 2 + lane) << 16;
      } else {
        rope[e] = __ldg(reinterpret_cast<const uint32_t*>(row + kDv * 2) + lane);
      }
    }
    if (i == 0) to = row_of(spot, L, tab, status);
#pragma unroll
    for (int e = 0; e < kRowAhead; ++e) {
      const int64_t r = __shfl_sync(0xffffffffu, to, i + e), ap = __shfl_sync(0xffffffffu, angle_pos, i + e);
      if (in.gamma) {
        float v[8], sum = 0.f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          unpack8(x[e][j], v);
          sum = square8(v, sum);
        }
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
        const float inv = rsqrtf(sum * (1.f / kDv) + in.eps);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          unpack8(x[e][j], v);
          float g[8];
#pragma unroll
          for (int h = 0; h < 2; ++h)
            *reinterpret_cast<float4*>(g + 4 * h) = *reinterpret_cast<const float4*>(gamma_s + 128 * (2 * j + h) + 4 * lane);
          scale8(v, inv, g);
          x[e][j] = pack8(v);
        }
      }
      if (in.inv_freq) {
        const Turn t = turn_of(step, ap);
        const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&rope[e]));
        const __nv_bfloat162 o =
            __floats2bfloat162_rn(fmaf(f.x, t.c, -f.y * t.s), fmaf(f.x, t.s, f.y * t.c));
        rope[e] = *reinterpret_cast<const uint32_t*>(&o);
      }
      const Row out(x[e]);  // every lane's part: the row's groups are two lanes'
      if (!live[e] || r < 0) continue;
      unsigned char* row = arena + r * Row::kBytes;
      out.store(row, lane);
      unsigned char* end = row + Row::kRopeAt;
      if (in.halves) {
        unsigned short* d = reinterpret_cast<unsigned short*>(end);
        d[lane] = (unsigned short)rope[e];
        d[kRope / 2 + lane] = (unsigned short)(rope[e] >> 16);
      } else {
        reinterpret_cast<uint32_t*>(end)[lane] = rope[e];
      }
    }
  }
}

bool norm_args_ok(const void* gamma, int32_t gamma_dtype, float eps, int32_t rope_style) {
  return (gamma_dtype == DCP_F32 || gamma_dtype == DCP_BF16) && eps >= 0.f && eps < INFINITY &&
         !(reinterpret_cast<uintptr_t>(gamma) & 15) && (rope_style == DCP_ROPE_PAIRS || rope_style == DCP_ROPE_HALVES);
}

template <class Row>
int32_t norm_rope_append(const dcp_layout_t* layout, int32_t shard_begin, int32_t shard_end, const void* kv,
                         int64_t kv_stride, const void* gamma, int32_t gamma_dtype, float eps, const float* inv_freq,
                         int32_t rope_style, const int64_t* rope_pos, const int64_t* pos, const int32_t* req, int64_t T,
                         const int32_t* block_table, int32_t B, int64_t bt_stride, int64_t max_pages, void* arena,
                         int64_t pool_pages, int32_t* status, void* stream) {
  if (!cache_args_ok(layout, shard_begin, shard_end, T, B, bt_stride, max_pages, pool_pages) ||
      !norm_args_ok(gamma, gamma_dtype, eps, rope_style) || kv_stride < kDk || kv_stride % 8)
    return DCP_ERR_INVALID;
  if (T == 0) return DCP_OK;
  if (!kv || !pos || !req || !block_table || !arena || misaligned(kv, arena)) return DCP_ERR_INVALID;
  const int per_warp = tokens_per_warp(T);
  const int64_t blocks = token_blocks(T, per_warp);
  if (blocks > INT32_MAX || kv_stride > INT64_MAX / 4 / T) return DCP_ERR_UNSUPPORTED;
  const RowArgs in{static_cast<const unsigned char*>(kv), kv_stride * 2, gamma, gamma_dtype == DCP_BF16, eps, inv_freq,
                   rope_style == DCP_ROPE_HALVES, rope_pos};
  norm_rope_store_kernel<Row><<<(unsigned)blocks, kThreads, 0, as_stream(stream)>>>(
      to_layout(layout), shard_begin, shard_end, in, pos, req, T, per_warp,
      Table{block_table, B, bt_stride, max_pages, pool_pages}, static_cast<unsigned char*>(arena), status);
  return launch_status();
}

}  // namespace

