// dcp_norm_rope.cu — what lies between a projection's output and the cache or the
// absorption product: RMS norm of a row and rotation of its position dims, in one pass.
//
//   y_d = x_d * rsqrt(mean x^2 + eps) * gamma_d       (f32; without gamma: y = x)
//   (a, b) -> (a cos t - b sin t, a sin t + b cos t)  for each of the 32 pairs of the
//             64 position dims, t = position * inv_freq[i]
// and one rounding to bf16 at the end.
//
// Angles.  A position times a frequency in f32 is off by 0.03 rad at 10^6, and f64 is
// slow on this card (2 operations a clock and SM).  So a block turns the frequencies
// into steps of 2^-64 turns once, in f64, and a position's angle is one wrapping 64-bit
// product: the fraction of a turn to 2^-64 * position.  The step itself is off by
// 1.5 * 2^-53 of its value, 2e-10 rad at 10^6 rad.
//
// dcp_q_norm_rope: 8 lanes a row of 192 dims (three 16-byte accesses a lane, 128 bytes
// of each row side by side), 4 rows a warp step; a warp serves heads of one token, so
// that it computes the token's sines once.
// dcp_kv_norm_rope_append(_q4): a warp a token at a time, dims as store_q4_kernel has
// them; the row is never written anywhere but into its pool.
#include "dcp_rows.cuh"

namespace {

constexpr int kQDims = 192, kRope = kDk - kDv;  // 128 content + 64 position dims a head

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
  sincospif((float)(int32_t)(f >> 32) * 0x1p-31f, &t.s, &t.c);  // half turns in [-1, 1]
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

// What a block's tokens share, in shared memory: norm weights (f32 or bf16) in f32, and the frequencies' steps (f64 runs
// at 2 operations a clock and SM: once a block, not once a warp).
__device__ __forceinline__ void load_shared(const void* gamma, int bf16, int dims, float* g, const float* inv_freq,
                                            uint64_t* steps) {
  if (gamma)
    for (int i = threadIdx.x; i < dims; i += blockDim.x)
      g[i] = bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(gamma)[i]) : static_cast<const float*>(gamma)[i];
  if (inv_freq && threadIdx.x < kRope / 2) steps[threadIdx.x] = turn_step(__ldg(inv_freq + threadIdx.x));
  __syncthreads();
}

// 8 normed values: x * inv * gamma.
__device__ __forceinline__ void scale8(float (&v)[8], float inv, const float* g) {
  const float4 a = *reinterpret_cast<const float4*>(g), b = *reinterpret_cast<const float4*>(g + 4);
  v[0] = v[0] * inv * a.x; v[1] = v[1] * inv * a.y; v[2] = v[2] * inv * a.z; v[3] = v[3] * inv * a.w;
  v[4] = v[4] * inv * b.x; v[5] = v[5] * inv * b.y; v[6] = v[6] * inv * b.z; v[7] = v[7] * inv * b.w;
}

__device__ __forceinline__ float square8(const float (&v)[8], float sum) {
#pragma unroll
  for (int k = 0; k < 8; ++k) sum = fmaf(v[k], v[k], sum);
  return sum;
}

// ---------------------------------------------------------------- queries
constexpr int kQThreads = 256;

// Warp task: token task / parts, its heads [part * per, part * per + per).  The next step's row is on its way while
// this one's is worked on; sines lie in shared memory (an angle is computed once a warp, by lane `pair`).
template <bool kHalves>
__global__ void __launch_bounds__(kQThreads, 4) q_norm_rope_kernel(int64_t T, int32_t H, int32_t per, int32_t parts,
                                                                   const __nv_bfloat16* q, int64_t stride,
                                                                   const int64_t* __restrict__ pos, const void* gamma,
                                                                   int gamma_bf16, float eps,
                                                                   const float* __restrict__ inv_freq,
                                                                   __nv_bfloat16* out, int32_t* status) {
  __shared__ __align__(16) float gamma_s[kQDims];
  __shared__ uint64_t steps_s[kRope / 2];
  __shared__ __align__(16) float2 turn_s[kQThreads / 32][kRope / 2];
  const int64_t task = blockIdx.x * (int64_t)(kQThreads / 32) + (threadIdx.x >> 5);
  const int64_t t = parts == 1 ? task : (int64_t)((uint64_t)task / (uint32_t)parts);
  const int lane = threadIdx.x & 31, l = lane & 7;  // lane of its row: dims 64 j + [8 l, 8 l + 8), j < 3
  const int h0 = (int)(task - t * parts) * per, h1 = min(h0 + per, H);
  const __nv_bfloat16* src = q + (t * H + h0 + (lane >> 3)) * stride + 8 * l;
  uint4 x[3];
  auto load = [&](int h) {
#pragma unroll
    for (int j = 0; j < 3; ++j)
      x[j] = h < h1 ? *reinterpret_cast<const uint4*>(src + 64 * j) : make_uint4(0, 0, 0, 0);
    src += 4 * stride;
  };
  int h = h0 + (lane >> 3);
  int64_t p = -1;
  if (t < T) {
    p = __ldg(pos + t);
    load(h);
  }
  load_shared(gamma, gamma_bf16, kQDims, gamma_s, inv_freq, steps_s);
  if (p < 0) {
    if (t < T && p != -1 && lane == 0) flag(status, DCP_STATUS_BAD_POSITION);
    return;
  }
  if (inv_freq) {
    const Turn turn = turn_of(steps_s[lane], p);
    turn_s[threadIdx.x >> 5][lane] = make_float2(turn.s, turn.c);
    __syncwarp();
  }
  // pairs (2 i, 2 i + 1) lie in one lane, halves (i, i + 32) in lanes l and l ^ 4
  const float4* turns = reinterpret_cast<const float4*>(turn_s[threadIdx.x >> 5] + (kHalves ? 8 * (l & 3) : 4 * l));
  __nv_bfloat16* dst = out + (t * H + h) * (int64_t)kQDims + 8 * l;
  for (; h - (lane >> 3) < h1; h += 4) {
    uint4 y[3] = {x[0], x[1], x[2]};
    load(h + 4);
    float r = 1.f, v[8];
    if (gamma) {
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 3; ++j) {
        unpack8(y[j], v);
        sum = square8(v, sum);
      }
#pragma unroll
      for (int s = 1; s < 8; s <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
      r = rsqrtf(sum * (1.f / kQDims) + eps);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        unpack8(y[j], v);
        scale8(v, r, gamma_s + 64 * j + 8 * l);
        y[j] = pack8(v);
      }
    }
    unpack8(y[2], v);
    if (gamma) scale8(v, r, gamma_s + 128 + 8 * l);
    if (inv_freq) {
#pragma unroll
      for (int k = 0; k < (kHalves ? 4 : 2); ++k) {
        const float4 sc = turns[k];  // sine, cosine of two angles
        if (kHalves) {
          const float a = __shfl_xor_sync(0xffffffffu, v[2 * k], 4), b = __shfl_xor_sync(0xffffffffu, v[2 * k + 1], 4);
          v[2 * k] = fmaf(v[2 * k], sc.y, l < 4 ? -a * sc.x : a * sc.x);
          v[2 * k + 1] = fmaf(v[2 * k + 1], sc.w, l < 4 ? -b * sc.z : b * sc.z);
        } else {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float s = e ? sc.z : sc.x, c = e ? sc.w : sc.y, a = v[4 * k + 2 * e], b = v[4 * k + 2 * e + 1];
            v[4 * k + 2 * e] = fmaf(a, c, -b * s);
            v[4 * k + 2 * e + 1] = fmaf(a, s, b * c);
          }
        }
      }
    }
    y[2] = pack8(v);
    if (h < h1)
#pragma unroll
      for (int j = 0; j < 3; ++j) *reinterpret_cast<uint4*>(dst + 64 * j) = y[j];
    dst += 4 * kQDims;
  }
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

// Tokens whose loads are in flight before their stores: 32768 tokens take 14.9 us with 2 and four blocks an SM, 16.1 with
// 4 and two blocks, 18.4 with 3 and three; 16.0 with 1 and five.
constexpr int kRowAhead = 2;

template <bool kQ4>
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
  load_shared(in.gamma, in.gamma_bf16, kDv, gamma_s, in.inv_freq, steps_s);
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
          scale8(v, inv, gamma_s + 256 * j + 8 * lane);
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
      float2 top;
      if (kQ4) {  // largest magnitudes of this lane's two groups: its own 8 dims and its neighbour's
        const __nv_bfloat162 mine = __nv_bfloat162(top8(x[e][0]), top8(x[e][1]));
        top = __bfloat1622float2(__hmax2_nan(mine, __shfl_xor_sync(0xffffffffu, mine, 1)));
      }
      if (!live[e] || r < 0) continue;
      unsigned char* row = arena + r * (kQ4 ? kQ4RowBytes : kDk * 2);
      unsigned char* end = row + (kQ4 ? kQ4RopeOff : kDv * 2);
      if (kQ4) {
        const uint32_t scales = __nv_cvt_float2_to_fp8x2(make_float2(seventh(top.x), seventh(top.y)), __NV_SATFINITE,
                                                         __NV_E4M3);
        const float2 s = q4_scales_f32(scales);
        reinterpret_cast<uint32_t*>(row)[lane] = codes8(x[e][0], s.x, top.x);
        reinterpret_cast<uint32_t*>(row)[32 + lane] = codes8(x[e][1], s.y, top.y);
        row[kQ4ScaleOff + 16 * (lane & 1) + (lane >> 1)] = (unsigned char)(lane & 1 ? scales >> 8 : scales);
      } else {
        reinterpret_cast<uint4*>(row)[lane] = x[e][0];
        reinterpret_cast<uint4*>(row)[32 + lane] = x[e][1];
      }
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

template <bool kQ4>
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
  norm_rope_store_kernel<kQ4><<<(unsigned)blocks, kThreads, 0, as_stream(stream)>>>(
      to_layout(layout), shard_begin, shard_end, in, pos, req, T, per_warp,
      Table{block_table, B, bt_stride, max_pages, pool_pages}, static_cast<unsigned char*>(arena), status);
  return launch_status();
}

}  // namespace

extern "C" int32_t dcp_q_norm_rope(int64_t T, int32_t H, const void* q, int64_t q_stride, const int64_t* pos,
                                   const void* gamma, int32_t gamma_dtype, float eps, const float* inv_freq,
                                   int32_t rope_style, void* out, int32_t* status, void* stream) {
  if (T < 0 || H < 1 || q_stride < kQDims || q_stride % 8 || !norm_args_ok(gamma, gamma_dtype, eps, rope_style))
    return DCP_ERR_INVALID;
  if (T == 0) return DCP_OK;
  if (!q || !pos || !out || misaligned(q, out)) return DCP_ERR_INVALID;
  if (q_stride > INT64_MAX / 4 / H / T) return DCP_ERR_UNSUPPORTED;
  // Heads a warp takes of its token: all of them once that many warps fill the card, fewer (a multiple of a warp
  // step's 4) while they do not.
  int64_t parts = 1;
  const int64_t most = (H + 3) / 4;
  while (parts < most && T * parts < 4864) parts *= 2;
  parts = parts < most ? parts : most;
  const int32_t per = (int32_t)((most + parts - 1) / parts) * 4;
  parts = (H + per - 1) / per;
  const int64_t blocks = (T * parts + kQThreads / 32 - 1) / (kQThreads / 32);
  if (blocks > INT32_MAX) return DCP_ERR_UNSUPPORTED;
  const auto kernel = rope_style == DCP_ROPE_HALVES ? q_norm_rope_kernel<true> : q_norm_rope_kernel<false>;
  kernel<<<(unsigned)blocks, kQThreads, 0, as_stream(stream)>>>(
      T, H, per, (int32_t)parts, static_cast<const __nv_bfloat16*>(q), q_stride, pos, gamma, gamma_dtype == DCP_BF16, eps,
      inv_freq, static_cast<__nv_bfloat16*>(out), status);
  return launch_status();
}

extern "C" int32_t dcp_kv_norm_rope_append(const dcp_layout_t* layout, int32_t shard_begin, int32_t shard_end,
                                           const void* kv, int64_t kv_stride, const void* gamma, int32_t gamma_dtype,
                                           float eps, const float* inv_freq, int32_t rope_style,
                                           const int64_t* rope_pos, const int64_t* pos, const int32_t* req, int64_t T,
                                           const int32_t* block_table, int32_t B, int64_t bt_stride, int64_t max_pages,
                                           void* arena, int64_t pool_pages, int32_t* status, void* stream) {
  return norm_rope_append<false>(layout, shard_begin, shard_end, kv, kv_stride, gamma, gamma_dtype, eps, inv_freq,
                                 rope_style, rope_pos, pos, req, T, block_table, B, bt_stride, max_pages, arena,
                                 pool_pages, status, stream);
}

extern "C" int32_t dcp_kv_norm_rope_append_q4(const dcp_layout_t* layout, int32_t shard_begin, int32_t shard_end,
                                              const void* kv, int64_t kv_stride, const void* gamma,
                                              int32_t gamma_dtype, float eps, const float* inv_freq,
                                              int32_t rope_style, const int64_t* rope_pos, const int64_t* pos,
                                              const int32_t* req, int64_t T, const int32_t* block_table, int32_t B,
                                              int64_t bt_stride, int64_t max_pages, void* arena, int64_t pool_pages,
                                              int32_t* status, void* stream) {
  return norm_rope_append<true>(layout, shard_begin, shard_end, kv, kv_stride, gamma, gamma_dtype, eps, inv_freq,
                                rope_style, rope_pos, pos, req, T, block_table, B, bt_stride, max_pages, arena,
                                pool_pages, status, stream);
}
