// dcp_decode_q4_few.cuh — the 4-bit partial decode of requests with at most 16 query
// rows (q_len * H).  Included by dcp_decode_q4.cu.
//
// With few rows the pair kernel's tile loop, a chain of exchanges that does not get
// shorter with fewer rows, takes 4 times as long as HBM.  Here one CTA takes whole rows,
// so nothing is exchanged between CTAs, and the codes go from shared memory straight to
// operands in registers: no dequantised tile is ever stored.  The products are warp-level
// m16n8k16 (2.15 cycles each an SM); of a tcgen05 product's 128 rows 7/8 would be padding,
// and its operand would have to be written to shared memory first.
//
// Per 64-key tile:
//   1. warp w: scores of keys [8 w, 8 w + 8) over all 576 dims (A: the query, prepared in
//      operand order; B: the codes of a key, 16 dims a lane), their row maxima;
//   2. every warp: the rows' maxima over all keys, the same in all; P = 2^(s - m) of its
//      keys, as bf16, to shared memory;
//   3. warp w: O dims [64 w, 64 w + 64) += P V over all keys (B: the codes of 8 dims of
//      two keys a lane, paired by key with a byte permute before they are dequantised).
// Both products leave the order of dims and keys free, as long as both operands use the
// same; the orders here make every load of the codes a run of 8 or 4 bytes without bank
// conflicts at the row stride of 416 bytes, and P's pairs adjacent.
//
// Measured with 8 rows against the pair kernel, us (calls in a captured graph, caches of
// quantised N(0, 1) rows): 32 requests of 64k tokens 383 / 533, 32 of 4k 43 / 66, 64 of 2k
// 45 / 76, 16 of 1k 20 / 33; one request of 64k 34 / 39, of 8k 20.5 / 22.5, of 1k 22.5 /
// 20.5.  Bound by its own instructions: 55 % of the issue slots with 16 warps an SM,
// shared-memory loads 55 %.
// Variants, on a cache of zeros.  Two tiles a step share the query's operands, 367 against
// 381 for the longest, but hold the ring's slots longer: 46 against 45 and 21 against 18.5
// for the short ones.  With two sets of 16 rows (two slots, the first warp loading) 32 rows
// took 27 against the pair kernel's 34 for 16 requests of 1k tokens, but 28 against 20 for
// one of 1k and 338 against 310 for 32 of 32k: 17 rows and more take the pair kernel.
namespace {

constexpr int kFewRows = 16;                       // most query rows
constexpr int kFewWarps = 8;                       // + one that loads
constexpr int kFewThreads = 32 * (kFewWarps + 1);
constexpr int kFewStages = 3;
constexpr int kFewStageBytes = kTile * kQ4RowBytes;
constexpr int kFewSteps = kDk / 16;                // k16 products of a score
constexpr int kFewPRow = kTile * 2 + 32;           // bytes of a row of P, padded

struct FewSmem {
  alignas(128) unsigned char ring[kFewStages][kFewStageBytes];
  uint4 q[kFewSteps][32];                          // A operands of the scores
  alignas(16) unsigned char p[kFewRows * kFewPRow];
  alignas(16) float wmax[kFewRows][kFewWarps];     // the warps' row maxima
  alignas(16) float lsum[kFewRows][kFewWarps];     // their row sums
  uint64_t full[kFewStages], empty[kFewStages];
  uint64_t live[kFewStages];                       // rows of the tile that count
  int abort;
};

__device__ __forceinline__ void few_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kFewWarps) : "memory"); }

__device__ __forceinline__ void mma_16816(float (&c)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

// Two e4m3 scales as one bf16 pair, and -136 times it (exact, as in q4_scales).
__device__ __forceinline__ void few_scale_pair(uint32_t two, uint32_t& s, uint32_t& off) {
  const float2 f = q4_scales_f32(two);
  const __nv_bfloat162 p = __floats2bfloat162_rn(f.x, f.y);
  const __nv_bfloat162 o = __hmul2(p, __float2bfloat162_rn(-136.f));
  s = *reinterpret_cast<const uint32_t*>(&p);
  off = *reinterpret_cast<const uint32_t*>(&o);
}

__global__ void __launch_bounds__(kFewThreads, 2) few_q4_kernel(const unsigned char* __restrict__ arena, TcArgs a) {
  extern __shared__ __align__(128) unsigned char few_smem[];
  FewSmem& sm = *reinterpret_cast<FewSmem*>(few_smem);
  griddep_wait();  // nothing the plan kernel wrote is read before this
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  const int v = blockIdx.x;
  const int32_t U = a.B * a.n_held;
  const int64_t T = a.tile_start[U];
  const int64_t lo = range_lo(T, v, a.V), hi = range_lo(T, v + 1, a.V);
  volatile int* abort_s = &sm.abort;
  if (tid == 0) {
    sm.abort = 0;
    for (int i = 0; i < kFewStages; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], kFewWarps);
    }
    fence_barrier_init();
  }
  __syncthreads();
  if (lo >= hi) return;

  if (w == kFewWarps) {
    // ------------------------------------------------------------------ loader
    const int nbox = kTile / a.box_rows;
    const int32_t P = (int32_t)a.L.P;
    uint32_t m = 0, phase = 0;
    SegIter it;
    it.init(a.tile_start, U, lo, hi);
    int32_t u, t0, nt, kslot;
    bool whole, ok = true;
    while (ok && it.next(&u, &t0, &nt, &whole, &kslot)) {
      const int64_t nvis = unit_rows(a, u);
      const int32_t pool0 = u % a.n_held * (int32_t)a.pool_rows;
      const int32_t* table = a.bt + (int64_t)(u / a.n_held) * a.bt_stride;
#pragma unroll 1
      for (int32_t tile = t0; tile < t0 + nt; ++tile) {
        // lane: first pool row of its box, -1 past the length or on a bad page
        const int32_t rho = tile * kTile + lane * a.box_rows;
        int32_t y = -1, rows = 0;
        if (lane < nbox && rho < nvis) {
          const int32_t pidx = rho / P;
          const int32_t page = pidx < a.max_pages ? __ldg(table + pidx) : -1;
          if (page >= 0 && page < a.pool_pages) {
            y = pool0 + page * P + rho % P;
            rows = (int32_t)min(nvis - rho, (int64_t)a.box_rows);
          } else {
            flag(a.status, DCP_STATUS_BAD_PAGE_ID);
          }
        }
        const uint64_t mine = (rows == 64 ? ~0ull : (1ull << rows) - 1) << ((lane * a.box_rows) & 63);
        const uint32_t live0 = __reduce_or_sync(0xffffffffu, (uint32_t)mine);
        const uint32_t live1 = __reduce_or_sync(0xffffffffu, (uint32_t)(mine >> 32));
        const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, y >= 0));
        const uint32_t bytes = (uint32_t)a.box_rows * kQ4RowBytes;
        if (!all_wait(&sm.empty[m], phase ^ 1, abort_s)) { ok = false; break; }
        if (lane == 0) {
          sm.live[m] = (uint64_t)live1 << 32 | live0;
          mbar_arrive_expect_tx(&sm.full[m], boxes * bytes);
        }
        __syncwarp();
        if (y >= 0)
          bulk_load(sm.ring[m] + lane * bytes, arena + (int64_t)y * kQ4RowBytes, bytes, &sm.full[m]);
        if (++m == kFewStages) {
          m = 0;
          phase ^= 1;
        }
      }
    }
  } else {
    // ------------------------------------------------------------------ products and softmax
    const int g = lane >> 2, t = lane & 3;
    // keys of this thread's score columns 2 t and 2 t + 1, of an 8-key block, and of its B column g
    const int key0 = t, key1 = 4 + (t ^ 2);
    const int key_b = (g & 1) ? 4 + ((g >> 1) ^ 2) : g >> 1;
    const uint32_t ring = smem_u32(sm.ring), q_s = smem_u32(sm.q) + lane * 16;
    const uint32_t qk_row = (uint32_t)(8 * w + key_b) * kQ4RowBytes;            // the key of the scores' B operand
    const uint32_t p_write = smem_u32(sm.p) + (uint32_t)g * kFewPRow + ((w >> 1) * 16 + t * 4 + 2 * (w & 1)) * 2;
    const uint32_t p_read = smem_u32(sm.p) + (uint32_t)g * kFewPRow + t * 8;
    const uint32_t pv_off = (uint32_t)key0 * kQ4RowBytes, pv_off1 = (uint32_t)key1 * kQ4RowBytes;
    const uint32_t scale_sel = (uint32_t)(t | (4 + t) << 4);                    // byte t of two words
    uint32_t m = 0, phase = 0;
    SegIter it;
    it.init(a.tile_start, U, lo, hi);
    int32_t u, t0, nt, kslot, cur_b = -1;
    bool whole;
    while (it.next(&u, &t0, &nt, &whole, &kslot)) {
      const int b = u / a.n_held, rs = u % a.n_held;
      const int64_t S = a.seq_lens[b];
      if (b != cur_b) {
        few_sync();  // the last request's query has been read
        for (int i = tid; i < kFewSteps * 32; i += 32 * kFewWarps) {
          const int step = i >> 5, ql = i & 31, qt = ql & 3;
          const int d = step < 32 ? 16 * (qt + 4 * (step >> 2)) + 4 * (step & 3)
                                  : kDv + 8 * (qt + 4 * ((step - 32) >> 1)) + 4 * (step & 1);
          uint2 r[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int row = (ql >> 2) + 8 * h;
            r[h] = row < a.R_total
                       ? __ldg(reinterpret_cast<const uint2*>(a.q + ((int64_t)b * a.R_total + row) * kDk + d))
                       : make_uint2(0, 0);
          }
          sm.q[step][ql] = make_uint4(r[0].x, r[1].x, r[0].y, r[1].y);
        }
        few_sync();
        cur_b = b;
      }
      int32_t lim[2];  // keys of tile t0 on that rows g and g + 8 see
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = g + 8 * h;
        lim[h] = row < a.R_total && S >= a.q_len
                     ? (int32_t)(rows_below(a, rs, S - a.q_len + row / a.H + 1) - (int64_t)t0 * kTile)
                     : 0;
      }
      float o[8][4];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
      float m_ref[2] = {kNoRef, kNoRef}, l[2] = {0.f, 0.f};
#pragma unroll 1
      for (int jj = 0; jj < nt; ++jj) {
        // (after an abort every wait returns at once, so that all warps meet at the barriers)
        all_wait(&sm.full[m], phase, abort_s);
        const uint32_t tile_s = ring + m * kFewStageBytes;
        const uint64_t live = sm.live[m];
        // ---- scores of 8 keys, even and odd products apart (a chain of 18)
        float s2c[2][4];
#pragma unroll
        for (int e = 0; e < 2; ++e) s2c[e][0] = s2c[e][1] = s2c[e][2] = s2c[e][3] = 0.f;
        const uint4 sc[2] = {ld_shared_v4(tile_s + qk_row + kQ4ScaleOff), ld_shared_v4(tile_s + qk_row + kQ4ScaleOff + 16)};
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          uint32_t s2[2], off2[2];
          const uint4& x4 = sc[i >> 2];
          const uint32_t w0 = (i & 2) ? x4.z : x4.x, w1 = (i & 2) ? x4.w : x4.y;
          q4_scales(__byte_perm(w0, w1, scale_sel), s2, off2);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float2 c = ld_shared_f32x2(tile_s + qk_row + 8 * t + 32 * (i + k));
            const uint32_t code[2] = {__float_as_uint(c.x), __float_as_uint(c.y)};
#pragma unroll
            for (int word = 0; word < 2; ++word) {
              const int step = (i + k) * 4 + word * 2;
              const uint4 qa = ld_shared_v4(q_s + 512 * step), qb = ld_shared_v4(q_s + 512 * (step + 1));
              uint32_t x[4];
              q4_values(code[word], s2[k], off2[k], x);
              mma_16816(s2c[0], qa, x[0], x[1]);
              mma_16816(s2c[1], qb, x[2], x[3]);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint4 qa = ld_shared_v4(q_s + 512 * (32 + 2 * i)), qb = ld_shared_v4(q_s + 512 * (33 + 2 * i));
          const uint4 x = ld_shared_v4(tile_s + qk_row + kQ4RopeOff + 16 * t + 64 * i);
          mma_16816(s2c[0], qa, x.x, x.y);
          mma_16816(s2c[1], qb, x.z, x.w);
        }
        float s[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) s[c] = s2c[0][c] + s2c[1][c];
        // ---- masks, row maxima
        if (live != ~0ull || min(lim[0], lim[1]) < kTile) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int key = 8 * w + (c & 1 ? key1 : key0);
            if (key >= lim[c >> 1] || !(live >> key & 1)) s[c] = -INFINITY;
          }
          // a row that does not count is 0 in P V, whatever its bytes are: its scales become 0
          const int key = 8 * w + (lane >> 2);
          if (!(live >> key & 1))
            asm volatile("st.shared.v2.b32 [%0], {%1, %1};" ::"r"(tile_s + key * kQ4RowBytes + kQ4ScaleOff + 8 * t), "r"(0)
                         : "memory");
          fence_proxy_async_smem();  // before the next copy into the slot
        }
        float mx[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          mx[h] = fmax_nan(s[2 * h], s[2 * h + 1]);
          mx[h] = fmax_nan(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
          mx[h] = fmax_nan(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
          if (t == 0) sm.wmax[g + 8 * h][w] = mx[h];
          lim[h] -= kTile;
        }
        few_sync();
        // ---- P
        float alpha[2];
        bool raised = false, nan = false;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float4 x = *reinterpret_cast<const float4*>(&sm.wmax[g + 8 * h][0]);
          const float4 y = *reinterpret_cast<const float4*>(&sm.wmax[g + 8 * h][4]);
          const float mt =
              fmax_nan(fmax3_nan(fmax3_nan(x.x, x.y, x.z), x.w, y.x), fmax3_nan(y.y, y.z, y.w)) * a.scale_log2;
          alpha[h] = 1.f;
          if (!(mt <= m_ref[h] + kRescaleThreshold)) {  // also the row's first visible key, and NaN
            raised = true;
            if (mt == mt) {
              alpha[h] = exp2f(m_ref[h] - mt);
              m_ref[h] = mt;
            } else {
              nan = true;
            }
          }
        }
        if (__any_sync(0xffffffffu, raised)) {
          // A NaN scale has made its key's score NaN in every row that sees the key (the last row sees
          // every live key, so all warps meet it here); it becomes 0 for the rows that do not, whose
          // weight 0 a NaN value would still turn into NaN.
          if (__any_sync(0xffffffffu, nan)) {
            const uint32_t at = tile_s + (8 * w + (lane >> 2)) * kQ4RowBytes + kQ4ScaleOff + 8 * t;
            const float2 two = ld_shared_f32x2(at);
            const uint32_t lo = __float_as_uint(two.x), hi = __float_as_uint(two.y);
            // 0xFF in the bytes that are NaN (all bits below the sign set)
            const uint32_t bad_lo = __vcmpeq4(lo & 0x7F7F7F7Fu, 0x7F7F7F7Fu), bad_hi = __vcmpeq4(hi & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
            if (bad_lo | bad_hi) {
              st_shared_f32x2(at, __uint_as_float(lo & ~bad_lo), __uint_as_float(hi & ~bad_hi));
              fence_proxy_async_smem();  // before the next copy into the slot
            }
          }
          l[0] *= alpha[0];
          l[1] *= alpha[1];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            o[j][0] *= alpha[0];
            o[j][1] *= alpha[0];
            o[j][2] *= alpha[1];
            o[j][3] *= alpha[1];
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float p0 = fast_exp2(fmaf(s[2 * h], a.scale_log2, -m_ref[h]));
          const float p1 = fast_exp2(fmaf(s[2 * h + 1], a.scale_log2, -m_ref[h]));
          l[h] += p0 + p1;
          const __nv_bfloat162 pp = __floats2bfloat162_rn(p0, p1);
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(p_write + 8 * h * kFewPRow),
                       "r"(*reinterpret_cast<const uint32_t*>(&pp))
                       : "memory");
        }
        few_sync();
        // ---- O += P V, 16 keys a product
        const uint32_t codes = tile_s + 4 * (8 * w + g), scales = tile_s + kQ4ScaleOff + 4 * w + (g >> 1);
#pragma unroll
        for (int k16 = 0; k16 < 4; ++k16) {
          const float2 pa = ld_shared_f32x2(p_read + 32 * k16);
          const float2 pb = ld_shared_f32x2(p_read + 8 * kFewPRow + 32 * k16);
          const uint4 pf = make_uint4(__float_as_uint(pa.x), __float_as_uint(pb.x), __float_as_uint(pa.y),
                                      __float_as_uint(pb.y));
          uint32_t x[2][2][4];  // [key pair][dims 2 i, dims 2 i + 1][i]
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t k0 = (uint32_t)(16 * k16 + 8 * h) * kQ4RowBytes + pv_off;
            const uint32_t k1 = (uint32_t)(16 * k16 + 8 * h) * kQ4RowBytes + pv_off1;
            const uint32_t c0 = ld_shared_u32(codes + k0), c1 = ld_shared_u32(codes + k1);
            uint32_t sp, op;
            few_scale_pair(ld_shared_u8(scales + k0) | ld_shared_u8(scales + k1) << 8, sp, op);
            q4_values(__byte_perm(c0, c1, 0x5410), sp, op, x[h][0]);
            q4_values(__byte_perm(c0, c1, 0x7632), sp, op, x[h][1]);
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) mma_16816(o[j], pf, x[0][j & 1][j >> 1], x[1][j & 1][j >> 1]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.empty[m]);
        if (++m == kFewStages) {
          m = 0;
          phase ^= 1;
        }
      }
      // ---- epilogue: O / l, lse
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        if (t == 0) sm.lsum[g + 8 * h][w] = l[h];
      }
      few_sync();
      const int64_t out_base = ((int64_t)rs * a.B + b) * a.R_total;
      const int64_t piece_base = (int64_t)(2 * v + kslot) * a.R_total;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = g + 8 * h;
        if (row >= a.R_total) continue;
        const float4 x = *reinterpret_cast<const float4*>(&sm.lsum[row][0]);
        const float4 y = *reinterpret_cast<const float4*>(&sm.lsum[row][4]);
        const float l_row = ((x.x + x.y) + (x.z + x.w)) + ((y.x + y.y) + (y.z + y.w));
        const float inv = l_row != 0.f ? 1.f / l_row : 0.f;  // 0: no key seen; a NaN stays one
        const int d0 = 64 * w + 16 * t;
        if (whole && a.o_bf16) {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o_part) + (out_base + row) * kDv + d0);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t r[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const __nv_bfloat162 z = __floats2bfloat162_rn(o[2 * i][2 * h + c] * inv, o[2 * i + 1][2 * h + c] * inv);
              r[i] = *reinterpret_cast<const uint32_t*>(&z);
            }
            dst[c] = make_uint4(r[0], r[1], r[2], r[3]);
          }
        } else {
          float4* dst = reinterpret_cast<float4*>(
              (whole ? static_cast<float*>(a.o_part) + (out_base + row) * kDv : a.piece_o + (piece_base + row) * kDv) + d0);
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              dst[2 * c + i] = make_float4(o[4 * i][2 * h + c] * inv, o[4 * i + 1][2 * h + c] * inv,
                                           o[4 * i + 2][2 * h + c] * inv, o[4 * i + 3][2 * h + c] * inv);
        }
        if (w == 0 && t == 0) {
          const float lse2 = l_row != 0.f ? m_ref[h] + log2f(l_row) : -INFINITY;
          if (whole)
            a.lse_part[out_base + row] = a.base2 ? lse2 : lse2 * kLn2;
          else
            a.piece_lse[piece_base + row] = lse2;
        }
      }
    }
  }
  __syncthreads();
  if (*abort_s) {
    if (tid == 0) flag(a.status, DCP_STATUS_TIMEOUT);
    __nanosleep(100000);  // copies in flight land first
  }
}

}  // namespace
