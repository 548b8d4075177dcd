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
#include "dcp_norm_rope.cuh"

namespace {

constexpr int kQDims = 192;  // 128 content + 64 position dims a head

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
  return norm_rope_append<Bf16Row>(layout, shard_begin, shard_end, kv, kv_stride, gamma, gamma_dtype, eps, inv_freq,
                                 rope_style, rope_pos, pos, req, T, block_table, B, bt_stride, max_pages, arena,
                                 pool_pages, status, stream);
}
