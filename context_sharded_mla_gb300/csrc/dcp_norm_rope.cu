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
// product: the fraction of a turn to 2^-65 * position.  The step itself is off by
// 1.5 * 2^-53 of its value, 2e-10 rad at 10^6 rad.  Sine and cosine of half turns, to a last
// place: the hardware's take radians and are off by up to 2^-21, which shows where a rotated
// value is small beside its pair, for 1 % of the append's time (18.9 against 18.8 us).
//
// dcp_q_norm_rope: 8 lanes a row of 192 dims, 48 bytes each, 4 rows a warp step; a warp
// serves heads of one token, so that it computes the token's sines once.  Memory-bound:
// 768 bytes a row.
// dcp_kv_norm_rope_append(_q4): a warp a token at a time, dims as store_q4_kernel has
// them; the row is never written anywhere but into its pool.
#include "dcp_norm_rope.cuh"

namespace {

constexpr int kQDims = 192;  // 128 content + 64 position dims a head

// ---------------------------------------------------------------- queries
constexpr int kQThreads = 256;

// Lane l of a row's 8 has dims [8 l, 8 l + 8) of each 64.  For the rotation a lane wants whole pairs: of pairs
// (2 i, 2 i + 1) it has four, first to last; of halves (i, i + 32) it trades four dims with lane l ^ 4 (both ways as
// bf16), so that it has pairs first(l) .. first(l) + 3, their first dims in the low and their second in the high words.
template <bool kHalves>
struct Pairs {
  __device__ static int first(int l) { return !kHalves ? 4 * l : l < 4 ? 8 * l : 8 * (l - 4) + 4; }
  __device__ static uint4 in(const uint4& x, int l) {
    if (!kHalves) return x;
    const uint32_t a = __shfl_xor_sync(0xffffffffu, l < 4 ? x.z : x.x, 4), b = __shfl_xor_sync(0xffffffffu, l < 4 ? x.w : x.y, 4);
    return l < 4 ? make_uint4(x.x, x.y, a, b) : make_uint4(a, b, x.z, x.w);
  }
  __device__ static uint4 out(const uint4& x, int l) {
    if (!kHalves) return x;
    const uint32_t a = __shfl_xor_sync(0xffffffffu, l < 4 ? x.z : x.x, 4), b = __shfl_xor_sync(0xffffffffu, l < 4 ? x.w : x.y, 4);
    return l < 4 ? make_uint4(x.x, x.y, a, b) : make_uint4(a, b, x.z, x.w);
  }
  // where value k of the eight that in() gives lies in the 64 dims
  __device__ static int dim(int l, int k) { return kHalves ? first(l) + (k & 3) + 32 * (k >> 2) : 8 * l + k; }
};

// A lane's norm weights in registers, the last eight in the order of Pairs: as they are (bf16, half the registers) or f32.
template <bool kHalves, bool kBf16>
struct QGamma;
template <bool kHalves>
struct QGamma<kHalves, true> {
  uint4 g[3];
  __device__ void load(const void* gamma, int l) {
    const uint4* p = static_cast<const uint4*>(gamma) + l;
#pragma unroll
    for (int j = 0; j < 3; ++j) g[j] = __ldg(p + 8 * j);
    g[2] = Pairs<kHalves>::in(g[2], l);
  }
  __device__ void get(int j, float (&v)[8]) const { unpack8(g[j], v); }
};
template <bool kHalves>
struct QGamma<kHalves, false> {
  float g[3][8];
  __device__ void load(const void* gamma, int l) {
    const float* f = static_cast<const float*>(gamma);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      g[0][k] = f[8 * l + k];
      g[1][k] = f[64 + 8 * l + k];
      g[2][k] = f[128 + Pairs<kHalves>::dim(l, k)];
    }
  }
  __device__ void get(int j, float (&v)[8]) const {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = g[j][k];
  }
};

// Warp task: token task / parts, its heads [part * per, part * per + per).  The next step's row is on its way while
// this one's is worked on; a lane's weights and the sines of its four pairs stay in registers.  8192 tokens of 128 heads:
// 131 us (halves) and 129 (pairs), 6.2 TB/s; with weights and sines in shared memory and eight dims traded one by one 136,
// bound there.  Four blocks an SM (two with f32 weights); three take 133, two 144.
template <bool kHalves, bool kGammaBf16>
__global__ void __launch_bounds__(kQThreads, kGammaBf16 ? 4 : 2)
    q_norm_rope_kernel(int64_t T, int32_t H, int32_t per, int32_t parts, const __nv_bfloat16* q, int64_t stride,
                       const int64_t* __restrict__ pos, const void* gamma, float eps, const float* __restrict__ inv_freq,
                       __nv_bfloat16* out, int32_t* status) {
  using P = Pairs<kHalves>;
  __shared__ uint64_t steps_s[kRope / 2];
  const int64_t task = blockIdx.x * (int64_t)(kQThreads / 32) + (threadIdx.x >> 5);
  const int64_t t = parts == 1 ? task : (int64_t)((uint64_t)task / (uint32_t)parts);
  const int lane = threadIdx.x & 31, l = lane & 7;  // 8 lanes a row
  const int h0 = (int)(task - t * parts) * per, h1 = min(h0 + per, H);
  int h = h0 + (lane >> 3);
  const __nv_bfloat16* src = q + (t * H + h) * stride + 8 * l;
  __nv_bfloat16* dst = out + (t * H + h) * (int64_t)kQDims + 8 * l;
  uint4 x[3];
  auto load = [&](int head) {
#pragma unroll
    for (int j = 0; j < 3; ++j)
      x[j] = head < h1 ? *reinterpret_cast<const uint4*>(src + 64 * j) : make_uint4(0, 0, 0, 0);
    src += 4 * stride;
  };
  int64_t p = -1;
  if (t < T) {
    p = __ldg(pos + t);
    load(h);
  }
  load_steps(inv_freq, steps_s);
  __syncthreads();
  if (p < 0) {
    if (t < T && p != -1 && lane == 0) flag(status, DCP_STATUS_BAD_POSITION);
    return;
  }
  QGamma<kHalves, kGammaBf16> g;
  if (gamma) g.load(gamma, l);
  Turn turn[4];
  if (inv_freq) {  // an angle a lane, handed to the lanes that turn that pair
    const Turn mine = turn_of(steps_s[lane], p);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      turn[k].s = __shfl_sync(0xffffffffu, mine.s, P::first(l) + k);
      turn[k].c = __shfl_sync(0xffffffffu, mine.c, P::first(l) + k);
    }
  }
  for (; h - (lane >> 3) < h1; h += 4) {
    uint4 y[3] = {x[0], x[1], x[2]};
    load(h + 4);
    float r = 1.f, v[8], w[8];
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
        g.get(j, w);
        scale8(v, r, w);
        y[j] = pack8(v);
      }
    }
    unpack8(P::in(y[2], l), v);
    if (gamma) {
      g.get(2, w);
      scale8(v, r, w);
    }
    if (inv_freq) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float &a = v[kHalves ? k : 2 * k], &b = v[kHalves ? 4 + k : 2 * k + 1];
        const float u = a;
        a = fmaf(u, turn[k].c, -b * turn[k].s);
        b = fmaf(u, turn[k].s, b * turn[k].c);
      }
    }
    y[2] = P::out(pack8(v), l);
    if (h < h1)
#pragma unroll
      for (int j = 0; j < 3; ++j) *reinterpret_cast<uint4*>(dst + 64 * j) = y[j];
    dst += 4 * kQDims;
  }
}

}  // namespace

extern "C" int32_t dcp_q_norm_rope(int64_t T, int32_t H, const void* q, int64_t q_stride, const int64_t* pos,
                                   const void* gamma, int32_t gamma_dtype, float eps, const float* inv_freq,
                                   int32_t rope_style, void* out, int32_t* status, void* stream) {
  if (T < 0 || H < 1 || H > 65535 || q_stride < kQDims || q_stride % 8 || !norm_args_ok(gamma, gamma_dtype, eps, rope_style))
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
  const bool halves = rope_style == DCP_ROPE_HALVES, bf16 = gamma_dtype == DCP_BF16;
  const auto kernel = halves ? (bf16 ? q_norm_rope_kernel<true, true> : q_norm_rope_kernel<true, false>)
                             : (bf16 ? q_norm_rope_kernel<false, true> : q_norm_rope_kernel<false, false>);
  kernel<<<(unsigned)blocks, kQThreads, 0, as_stream(stream)>>>(
      T, H, per, (int32_t)parts, static_cast<const __nv_bfloat16*>(q), q_stride, pos, gamma, eps, inv_freq,
      static_cast<__nv_bfloat16*>(out), status);
  return launch_status();
}

extern "C" int32_t dcp_kv_norm_rope_append(const dcp_layout_t* layout, int32_t shard_begin, int32_t shard_end,
                                           const void* kv, int64_t kv_stride, const void* gamma, int32_t gamma_dtype,
                                           float eps, const float* inv_freq, int32_t rope_style,
                                           const int64_t* rope_pos, const int64_t* pos, const int32_t* req, int64_t T,
                                           const int32_t* block_table, int32_t B, int64_t bt_stride, int64_t max_pages,
                                           void* arena, int64_t pool_pages, int32_t* status, void* stream) {
  return norm_rope_append<Bf16Row>(layout, shard_begin, shard_end, kv, kv_stride, gamma, gamma_dtype, eps, inv_freq,
                                 rope_style, rope_pos, pos, req, T, block_table, B, bt_stride, max_pages, arena,
                                 pool_pages, status, stream);
}
