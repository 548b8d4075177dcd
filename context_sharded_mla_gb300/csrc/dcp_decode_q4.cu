// dcp_decode_q4.cu — per-shard partial attention over a latent cache held in 4
// bits (row format: dcp_internal.cuh).  The method, the outputs and the sources
// are dcp_decode.cu's; only the keys and values come from 416-byte rows.
//
// Mathematics: value of dim d < 512 = code_d * scale_{d / 16}, 3 bits and a sign
// times an e4m3's 4 significant bits: exact in bf16, so the bf16 products see the
// cached values themselves and nothing is rounded on the way in.
//
// What bounds it: at 416 bytes a row, 55 query rows already outweigh HBM (2176
// flop per row and key against 282 flop per byte), so a full set of heads is bound
// inside the SM.  Of the resources a 64-key tile needs for 128 rows, in cycles: the
// tensor pipe 1340 (18 products of N = 64 at 47, which is what any N <= 64 costs,
// and 4 of N = 256 at 123), the network between the CTAs of a pair 1230 (24.5 KB at
// the 20 bytes a cycle that copies to a peer's shared memory reach), shared memory
// about 1800; and each softmax warp has some 390 instructions to get through.
//
// Design: the 2-CTA pair of dcp_decode.cu (CTA r holds half of the 576 key dims and
// half of the value dims of every tile), with
//   - the softmax split by keys: CTA r runs it for keys [32 r, 32 r + 32) of a tile
//     only.  It sends its partial scores of the other 32 keys (16 KB) and the P of its
//     own (8 KB), where exchanging all partial scores would send 32 KB and do every
//     exponential twice;
//   - all four query chunks of a CTA in TMEM; of the QK product's A operands only the
//     32 rope dims are read from shared memory;
//   - four slots of dequantised tiles, and the raw codes of a tile coming by TMA into
//     a ring of their own;
//   - short loops: the roles' loops share the instruction caches.
// Measured, us for 64 requests of 128k tokens and 96 heads / 32 of 32k and 128 heads
// (a chain of calls): all partial scores exchanged and codes loaded to registers
// 2690 / 431; softmax split by keys 3320 / 477 while the kernel was 147 KB of code
// (its warps waited for instructions more than for anything else); 80 KB of code
// 2620 / 389; fewer instructions in the softmax 2390 / 374; products issued by an
// elected lane of a converged warp (370 ns for the 18, against 817 from a lane's own
// branch) 2270 / 358; the next query loaded in whole lines 2290 / 349; fewer conversions
// of scales and a shorter fixup 2285 / 343; bad pages and NaN told apart 2294 / 344.  Reading the
// peer's scores with loads from its shared memory instead of copies (65 bytes a cycle
// alone) held up the warps' other loads: 3160 / 456.
//
// Warps (480 threads):
//   0-7    softmax, exchange, epilogue (16 rows each, two threads per row)
//   8-11   dequantise: warp 8 + w turns rows [16 w, 16 w + 16) of a raw tile into
//          the 128-byte-swizzled bf16 chunks both products read; a row past the
//          request's length or on a bad page is written as zeros, and what the
//          softmax has to know of bad pages is marked.  Warp 8 also loads the
//          tile's rope dims (bf16 in the cache) by TMA.
//   12     producer: page table, raw tiles
//   13     QK issuer (and loader of the query's rope operand), TMEM owner
//   14     PV issuer
// TMEM: O [0, 256), S [256, 320), two P tiles [320, 384), query [384, 512).
#include "dcp_decode.cuh"

namespace {

constexpr int kSoftmaxWarps = 8;
constexpr int kDequantWarp0 = 8;
constexpr int kDequantWarps = 4;
constexpr int kDequantRows = kTile / kDequantWarps;
constexpr int kProducerWarp = 12;
constexpr int kMmaWarp = 13;                  // QK issuer and TMEM owner
constexpr int kPvWarp = 14;
constexpr int kThreads = 480;
constexpr int kMaxSlots = 4;                  // dequantised tiles
constexpr int kMaxRaw = 4;                    // raw tiles
constexpr int kL2Ahead = 3;                   // tiles between a tile's L2 prefetch and its raw load
constexpr int kRawCodeBytes = kTile * 128;    // this CTA's 256 dims, 128-byte swizzle
constexpr int kRawScaleBytes = kTile * 16;    // their 16 scales a row
constexpr int kRawBytes = kRawCodeBytes + kRawScaleBytes;
constexpr uint32_t kOCol = 0, kSCol = 256, kPCol = 320, kQCol = 384;
constexpr int kOwnKeys = kTile / 2;           // keys of a tile whose softmax this CTA runs
constexpr int kSRowBytes = kOwnKeys * 4;      // one row of the partial scores the peer needs
constexpr int kSWarpBytes = kHalfRows * kSRowBytes;
constexpr int kPOff = kHalfRows * kOwnKeys * 2;            // a warp's P message: P in bf16, then per row
constexpr int kPWarpBytes = kPOff + 2 * kHalfRows * 4;     // its reference and its sum
constexpr int kMaxBoxes = 8;                  // pages a tile can touch (page size >= 8)

struct SmemLayout {
  uint32_t qr, s, sbuf, p, pbuf, ring, raw, bars, rows, misc, total;
};

enum Bar { kQFull = 0, kQEmpty, kSFull, kSFree, kPFull, kPVDone = kPFull + 2, kOFree = kPVDone + 2,
           kSLand,                    // [2 buffers][8 channels]: the peer's partial scores of a warp's rows
           kPLand = kSLand + 16,      // [2 buffers][8 channels]: its P of those rows
           kTFull = kPLand + 16, kTEmpty = kTFull + kMaxSlots,   // dequantised tile slots
           kRFull = kTEmpty + kMaxSlots, kREmpty = kRFull + kMaxRaw, kNumBars = kREmpty + kMaxRaw };

// A raw tile's description, written by the producer before the tile's TMA copies.
struct RawRows {
  int32_t y[kMaxBoxes];  // first pool row of each box, -1: none (past the length, bad page)
  int32_t valid;         // rows of the tile below the request's length
};

__host__ __device__ inline SmemLayout smem_layout(int Rg, int nts, int nraw) {
  SmemLayout s;
  s.qr = 0;                                    // query rope dims [32 r, +32): [128][32] bf16, rows >= Rg zero
  s.s = 128 * 64;                              // two buffers of partial scores [Rg][32] fp32, staged / landed
  s.sbuf = (uint32_t)Rg * kSRowBytes;
  s.p = s.s + 2 * s.sbuf;                      // two buffers of P messages, staged / landed
  s.pbuf = (uint32_t)(Rg / kHalfRows) * kPWarpBytes;
  s.ring = round1024(s.p + 2 * s.pbuf);        // tile slots: 4 value chunks + this CTA's rope half
  s.raw = s.ring + nts * kSlotBytes;
  s.bars = s.raw + nraw * kRawBytes;
  s.rows = s.bars + kNumBars * 8;
  s.misc = (s.rows + kMaxRaw * (uint32_t)sizeof(RawRows) + 7u) & ~7u;
  s.total = s.misc + 64;
  return s;
}

// The loop of every role has to fit the instruction caches together with the
// others' (with everything inlined the kernel was 147 KB and its warps waited for
// instructions more than for anything else), so what runs rarely stays out of line:
// a wait that does not succeed at once, the 64-bit count of a unit's rows, the store
// of O rows, and what bad pages and NaN need.
__device__ __noinline__ bool wait_rest(uint64_t* bar, uint32_t parity, volatile int* abort_s) {
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait_for(bar, parity, kSuspendNs)) {
    if (*abort_s) return false;
    if (globaltimer() - t0 > kWaitLimitNs) {
      *abort_s = 1;
      return false;
    }
  }
  return true;
}

// A warp-uniform wait (false after an abort).
__device__ __forceinline__ bool all_wait(uint64_t* bar, uint32_t parity, volatile int* abort_s) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, wait_rest(bar, parity, abort_s));
}
// Rows of shard shard_begin + rs below position x, as far as the table goes (32-bit arithmetic where it
// does; a 64-bit division is some hundred instructions).
__device__ __noinline__ int64_t rows_below_long(const TcArgs& a, int rs, int64_t x) {
  return count_of(a.shard_begin + rs, x, a.L);
}
__device__ __forceinline__ int64_t rows_below(const TcArgs& a, int rs, int64_t x) {
  const int64_t span = a.L.N * a.L.I;
  if (((x | span) >> 31) != 0) return min(rows_below_long(a, rs, x), a.max_rows);
  const uint32_t I = (uint32_t)a.L.I, n = (uint32_t)x / (uint32_t)span;
  const int32_t rest = (int32_t)((uint32_t)x - n * (uint32_t)span) - (a.shard_begin + rs) * (int32_t)I;
  return min((int64_t)n * I + min(max(rest, 0), (int32_t)I), a.max_rows);
}
__device__ __forceinline__ int64_t unit_rows(const TcArgs& a, int32_t u) {
  const int64_t S = a.seq_lens[u / a.n_held];
  return S < a.q_len ? 0 : rows_below(a, u % a.n_held, S);
}

// Which of a dequantising warp's two 8-row groups of tile j are on a bad page (bits 0 and 1),
// or ~0 after an abort.  For a whole warp; out of line because only NaN scores ask for it.
__device__ __noinline__ uint32_t bad_groups(uint64_t* full, const unsigned char* flags, uint32_t j, uint32_t nts,
                                            volatile int* abort_s) {
  const uint32_t ts = j % nts;
  if (!all_wait(full + ts, (j / nts) & 1, abort_s)) return ~0u;  // has passed: the scores are there
  return flags[kDequantWarps * ts];
}

// NaN among eight e4m3 scales (all bits below the sign set): not 0.
__device__ __forceinline__ uint32_t e4m3_nans(uint32_t a, uint32_t b) {
  return (((a & 0x7F7F7F7Fu) + 0x01010101u) | ((b & 0x7F7F7F7Fu) + 0x01010101u)) & 0x80808080u;
}

// The NaN values of a tile become 0, by a whole warp, between the tile's two products.  A
// NaN scale has made the scores of its key NaN, and so the weight in every row that sees the
// key; a row that does not has weight 0, which a NaN value would still turn into NaN.
__device__ __noinline__ void zero_nan_values(uint32_t slot) {
#pragma unroll 1
  for (uint32_t at = slot + 16 * (threadIdx.x & 31); at < slot + kRopeOff; at += 512) {
    const uint4 v = ld_shared_v4(at);
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&w[i]);
      const uint32_t num = __heq2_mask(x, x);  // 0 in the half of a NaN
      w[i] &= num;
    }
    st_shared_v4(at, w[0], w[1], w[2], w[3]);
  }
  fence_proxy_async_smem();  // the tensor core reads the tile through the async proxy
  __syncwarp();
}

// No copy brings the rope dims of a bad page: NaN there makes the keys' scores NaN, which is
// what the softmax looks at the flags for.  For a whole warp: its two 8-row groups by `bad`.
__device__ __noinline__ void nan_rope(uint32_t at, uint32_t bad) {
#pragma unroll
  for (int e = 0; e < 2; ++e)
    if (bad >> e & 1) st_shared_v4(at + 512 * e + 16 * (threadIdx.x & 31), ~0u, ~0u, ~0u, ~0u);
}

constexpr float kNoRef = -1e30f;  // a row that has seen no key: 2^(s - kNoRef) is only formed for s = -inf

// 2^d for a whole number d <= 8, exactly; 0 below 2^-126.
__device__ __forceinline__ float pow2(float d) {
  return d >= -126.f ? __uint_as_float((uint32_t)((int)d + 127) << 23) : 0.f;
}

// bf16 pairs times a power of two (exact down to bf16's subnormals).
__device__ __forceinline__ void scale_bf16x2(uint32_t (&x)[8], float f) {
  const __nv_bfloat162 f2 = __float2bfloat162_rn(f);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&x[i]), f2);
    x[i] = *reinterpret_cast<const uint32_t*>(&r);
  }
}

// The 16 O rows of a softmax warp times `inv` -> the output rows (bf16 or fp32) or
// the fp32 piece rows; thread t holds dims [d0, d0 + 128) of row r0 + t % 16.  Rows
// below rows_here are written.  64 bytes of each half-row at a time go through
// `stage` (2 KB: row r's half h is segment 2 r + (h ^ r % 2), its 16-byte piece c
// at slot c ^ (r / 2) % 4), so that four lanes write one 64-byte run.
__device__ __noinline__ void store_rows_q4(const TcArgs& a, uint32_t o_addr, int rows_here, bool whole,
                                           int64_t out_base, int64_t piece_base, int r0, int d0, float inv,
                                           uint32_t stage) {
  const int lane = threadIdx.x & 31;
  const int h = lane >> 4, lr = lane & 15;
  const int dbase = d0 - 128 * h;                   // this CTA's first dim
  const bool bf16 = whole && a.o_bf16;
  unsigned char* const out = whole ? static_cast<unsigned char*>(a.o_part) + out_base * kDv * (bf16 ? 2 : 4)
                                   : reinterpret_cast<unsigned char*>(a.piece_o + piece_base * kDv);
  const int esize = bf16 ? 2 : 4, dims = 64 / esize;  // dims of a 64-byte run
  const uint32_t mine = stage + (uint32_t)(2 * lr + (h ^ (lr & 1))) * 64;
#pragma unroll 1
  for (int d = 0; d < 128; d += dims) {
    uint32_t w[16];
    if (bf16) {
      uint32_t rr[32];
      tmem_ld16x2_sync<128>(o_addr + d, rr);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        __nv_bfloat162 hh = __floats2bfloat162_rn(__uint_as_float(rr[2 * e]) * inv, __uint_as_float(rr[2 * e + 1]) * inv);
        w[e] = *reinterpret_cast<uint32_t*>(&hh);
      }
    } else {
      tmem_ld16x2_16_sync<128>(o_addr + d, w);
#pragma unroll
      for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) * inv);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c)
      st_shared_v4(mine + (uint32_t)((c ^ (lr >> 1)) & 3) * 16, w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int sg = 8 * i + (lane >> 2), c = lane & 3;
      const int sr = sg >> 1, sh = (sg ^ sr) & 1;
      const uint4 v = ld_shared_v4(stage + (uint32_t)sg * 64 + (uint32_t)((c ^ (sr >> 1)) & 3) * 16);
      if (r0 + sr < rows_here)
        *reinterpret_cast<uint4*>(out + ((int64_t)(r0 + sr) * kDv + dbase + 128 * sh + d) * esize + 16 * c) = v;
    }
    __syncwarp();                                   // the reads are done before the next run's writes
  }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    partial_q4_kernel(const __grid_constant__ CUtensorMap tmap_q64, const __grid_constant__ CUtensorMap tmap_code,
                      const __grid_constant__ CUtensorMap tmap_scale, const __grid_constant__ CUtensorMap tmap_rope,
                      const unsigned char* __restrict__ arena, TcArgs a) {
  extern __shared__ __align__(1024) unsigned char smem[];
  // The layout needs a 1024-byte aligned base: every CTA of the launch sees the
  // same base, so a misaligned one makes all of them stop, before any barrier.
  if ((smem_u32(smem) & 1023u) != 0) {
    if (threadIdx.x == 0) flag(a.status, DCP_STATUS_INTERNAL);
    return;
  }
  griddep_wait();  // nothing the plan kernel wrote is read before this
  const int nts = a.nts, nraw = a.nraw;
  const SmemLayout sl = smem_layout(a.Rg, nts, nraw);
  unsigned char* qr_s = smem + sl.qr;
  unsigned char* ring = smem + sl.ring;
  unsigned char* raw = smem + sl.raw;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + sl.bars);
  RawRows* raw_rows = reinterpret_cast<RawRows*>(smem + sl.rows);
  uint32_t* tmem_base_s = reinterpret_cast<uint32_t*>(smem + sl.misc);
  volatile int* abort_s = reinterpret_cast<volatile int*>(smem + sl.misc + 4);
  // [slot][dequantising warp], about the warp's 16 rows of the tile: bit e, its 8-row group e is on a
  // bad page; bit 2, a scale among them is NaN
  unsigned char* tile_flags = smem + sl.misc + 16;

  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  const int cid = blockIdx.x >> 1;  // cluster index
  const int v = cid / a.ngroups;
  const int g = cid % a.ngroups;
  const int Rg = a.Rg;
  int nsoft = 0;  // softmax warps with rows of the group (warp w < 8 serves rows 32 (w % 4) + 16 (w / 4) + [0, 16))
  for (int w = 0; w < kSoftmaxWarps; ++w) nsoft += 32 * (w & 3) + kHalfRows * (w >> 2) < Rg;
  const int32_t U = a.B * a.n_held;
  const int64_t T = a.tile_start[U];
  const int64_t lo = range_lo(T, v, a.V), hi = range_lo(T, v + 1, a.V);
  const uint32_t ntiles = (uint32_t)(hi - lo);

  if (tid == 0) {
    *abort_s = 0;
    for (int i = 0; i < kNumBars; ++i) mbar_init(&bars[i], 1);
    mbar_init(&bars[kQFull], nsoft + 1);  // softmax warps + the rope TMA
    mbar_init(&bars[kSFree], nsoft);
    for (int i = 0; i < 2; ++i) mbar_init(&bars[kPFull + i], nsoft);
    mbar_init(&bars[kOFree], nsoft);
    for (int i = 0; i < kMaxSlots; ++i) mbar_init(&bars[kTFull + i], kDequantWarps + 1);  // + the rope TMA
    for (int i = 0; i < kMaxRaw; ++i) mbar_init(&bars[kREmpty + i], kDequantWarps);
    fence_barrier_init();
    // tile j's messages from the peer land in buffer (j & 1) ^ 1: expect tiles 0 and 1
    // (what is expected after the last tile never comes, and nothing waits for it)
    for (int w = 0; w < 2 * kSoftmaxWarps; ++w) {
      mbar_arrive_expect_tx(&bars[kSLand + w], kSWarpBytes);
      mbar_arrive_expect_tx(&bars[kPLand + w], kPWarpBytes);
    }
  }
  // Rope rows that no copy brings (pages past a request's length) are multiplied
  // into scores that are masked: start from finite zeros.  Query rope rows past
  // the group stay zero for good, and so do their score lanes.
  for (int i = tid; i < nts * kSlotBytes / 16; i += kThreads) reinterpret_cast<uint4*>(ring)[i] = make_uint4(0, 0, 0, 0);
  for (int i = tid; i < 128 * 64 / 16; i += kThreads) reinterpret_cast<uint4*>(qr_s)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_base_s, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  cluster_sync();  // both CTAs' barriers exist before any remote store or arrive
  tc_fence_after();
  const uint32_t tmem = *tmem_base_s;

  if (warp == kProducerWarp) {
    // ------------------------------------------------------------------ producer
    // Raw tiles, as boxes of min(page size, 64) rows.  Lane l holds the pool row of
    // box l of a batch of 32 (the page ids of the next batch are in flight); lane 0
    // waits for a raw slot, writes the tile's rows and issues its copies.
    if (lo < hi) {
      if (lane == 0) {
        prefetch_tmap(&tmap_code);
        prefetch_tmap(&tmap_scale);
        prefetch_tmap(&tmap_rope);
      }
      const int nbox = kTile / a.box_rows;
      const int32_t P = (int32_t)a.L.P;
      uint32_t m = 0, mphase = 0;  // raw slot of the next tile and its use parity
      SegIter it;
      it.init(a.tile_start, U, lo, hi);
      int32_t u, t0, nt, kslot;
      bool whole;
      bool ok = true;
      bool have = it.next(&u, &t0, &nt, &whole, &kslot);
      int64_t nvis_next = have ? unit_rows(a, u) : 0;
      // page id of lane's box of the batch that starts at box x0 of the unit (-1: none)
      auto page_of = [&](int32_t uu, int32_t x0, int32_t x_end) -> int32_t {
        const int32_t rho = (x0 + lane) * a.box_rows;
        const int32_t pidx = rho / P;
        return x0 + lane < x_end && pidx >= 0 && pidx < a.max_pages
                   ? __ldg(a.bt + (int64_t)(uu / a.n_held) * a.bt_stride + pidx)
                   : -1;
      };
      int32_t page = have ? page_of(u, t0 * nbox, (t0 + nt) * nbox) : -1;
      while (ok && have) {
        const int64_t nvis = nvis_next;
        const int32_t x_first = t0 * nbox, x_end = (t0 + nt) * nbox;
        const int32_t pool0 = u % a.n_held * (int32_t)a.pool_rows;
        SegIter nx = it;
        int32_t u2 = 0, t02 = 0, nt2 = 0, ks2 = 0;
        bool wh2 = false;
        const bool has_next = nx.next(&u2, &t02, &nt2, &wh2, &ks2);
        int32_t y = -1;
#pragma unroll 1
        for (int32_t x = x_first; x < x_end; x += nbox) {
          const int32_t at = (x - x_first) & 31;
          if (at == 0) {
            // lane: first pool row of its box, -1 past the length or on a bad page; a box never
            // crosses a page: its height is min(P, 64) and it starts at a multiple of it
            const int32_t rho = (x + lane) * a.box_rows;
            y = -1;
            if (x + lane < x_end && rho < nvis) {
              if (page >= 0 && page < a.pool_pages)
                y = pool0 + page * P + rho % P;
              else if (rank == 0)
                flag(a.status, DCP_STATUS_BAD_PAGE_ID);
            }
            if (x + 32 < x_end) {
              page = page_of(u, x + 32, x_end);
            } else if (has_next) {
              page = page_of(u2, t02 * nbox, (t02 + nt2) * nbox);
              nvis_next = unit_rows(a, u2);
            }
          }
          if (!all_wait(&bars[kREmpty + m], mphase ^ 1, abort_s)) { ok = false; break; }
          const bool mine = lane >= at && lane < at + nbox;  // lanes of this tile's boxes
          if (mine) raw_rows[m].y[lane - at] = y;
          const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, mine && y >= 0));
          if (lane == 0) {
            const int64_t left = nvis - (int64_t)x * a.box_rows;
            raw_rows[m].valid = left < kTile ? (int32_t)left : kTile;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive_expect_tx(&bars[kRFull + m], boxes * a.box_rows * (128 + 16));
          __syncwarp();
          if (mine && y >= 0) {
            unsigned char* dst = raw + m * kRawBytes;
            const int q = (lane - at) * a.box_rows;
            tma_load_2d(dst + q * 128, &tmap_code, &bars[kRFull + m], 128 * (int)rank, y);
            tma_load_2d(dst + kRawCodeBytes + q * 16, &tmap_scale, &bars[kRFull + m], 16 * (int)rank, y);
            tma_prefetch_2d(&tmap_rope, kRopeHalf * (int)rank, y);  // loaded when its tile slot is free
          }
          // the same rows kL2Ahead tiles on, whole, into L2 (as far as this batch goes)
          if (lane >= at + kL2Ahead * nbox && lane < at + (kL2Ahead + 1) * nbox && y >= 0) {
            const int half = a.box_rows / 2;
            bulk_prefetch_l2(arena + (int64_t)(y + half * (int)rank) * kQ4RowBytes, half * kQ4RowBytes);
          }
          if (++m == (uint32_t)nraw) {
            m = 0;
            mphase ^= 1;
          }
        }
        it = nx;
        have = has_next;
        u = u2, t0 = t02, nt = nt2, whole = wh2, kslot = ks2;
      }
    }
  } else if (warp >= kDequantWarp0 && warp < kDequantWarp0 + kDequantWarps) {
    // ------------------------------------------------------------------ 4-bit rows -> bf16 tiles
    // Lane l serves row l % 8 of each of the warp's two 8-row groups (a group
    // never crosses a page) and the 32-dim pieces l / 8 and l / 8 + 4 of this
    // CTA's 256 dims; the 8 lanes of a shared-memory phase touch 8 different
    // swizzled 16-byte slots, on the way in and on the way out.
    const int w = warp - kDequantWarp0;
    const int r8 = lane & 7, pc = lane >> 3;
    const int nbox = kTile / a.box_rows;
    const int box0 = kDequantRows * w / a.box_rows, box1 = (kDequantRows * w + 8) / a.box_rows;
    uint32_t m = 0, mphase = 0, ts = 0, tphase = 0;
    bool ok = true;
    for (uint32_t j = 0; j < ntiles; ++j) {
      if (!all_wait(&bars[kRFull + m], mphase, abort_s)) { ok = false; break; }
      const RawRows& rr = raw_rows[m];
      const uint32_t src = smem_u32(raw) + m * kRawBytes;
      const int32_t y = lane < nbox ? rr.y[lane] : -1;  // lane q: first pool row of box q
      // the warp's 8-row groups that are below the length but on a bad page
      const uint32_t bad = (kDequantRows * w < rr.valid && rr.y[box0] < 0 ? 1u : 0u) |
                           (kDequantRows * w + 8 < rr.valid && rr.y[box1] < 0 ? 2u : 0u);
      // the tile's values, ready in registers before its slot is free
      uint32_t x[4][4][4], scales[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = kDequantRows * w + 8 * (e >> 1) + r8;
        const int piece = pc + 4 * (e & 1);  // of this CTA's 8
        const bool live = row < rr.valid && rr.y[e < 2 ? box0 : box1] >= 0;
        const uint4 code = ld_shared_v4(src + (uint32_t)row * 128 + (uint32_t)((piece ^ r8) << 4));
        const uint32_t two = ld_shared_u16(src + kRawCodeBytes + (uint32_t)row * 16 + 2 * piece);
        uint32_t s2[2], o2[2];
        scales[e] = two;
        q4_scales(live ? two : 0u, s2, o2);
        q4_values(code.x, s2[0], o2[0], x[e][0]);
        q4_values(code.y, s2[0], o2[0], x[e][1]);
        q4_values(code.z, s2[1], o2[1], x[e][2]);
        q4_values(code.w, s2[1], o2[1], x[e][3]);
      }
      // (rows that do not count may say so, too: their values are 0 already)
      const uint32_t nan = e4m3_nans(scales[0] | scales[1] << 16, scales[2] | scales[3] << 16);
      const uint32_t flags = bad | (__any_sync(0xffffffffu, nan != 0) ? 4u : 0u);
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kREmpty + m]);
      if (!all_wait(&bars[kTEmpty + ts], tphase ^ 1, abort_s)) { ok = false; break; }
      unsigned char* slot = ring + ts * kSlotBytes;
      if (w == 0) {
        const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, y >= 0));
        if (lane == 0) mbar_arrive_expect_tx(&bars[kTFull + ts], boxes * a.box_rows * 64);
        __syncwarp();
        if (y >= 0)
          tma_load_2d(slot + kRopeOff + lane * a.box_rows * 64, &tmap_rope, &bars[kTFull + ts], kRopeHalf * (int)rank, y);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int piece = pc + 4 * (e & 1);
        const uint32_t dst = smem_u32(slot) + (uint32_t)(piece >> 1) * kChunkBytes +
                             (uint32_t)(kDequantRows * w + 8 * (e >> 1) + r8) * 128;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          st_shared_v4(dst + (uint32_t)((4 * (piece & 1) + k) ^ r8) * 16, x[e][k][0], x[e][k][1], x[e][k][2], x[e][k][3]);
      }
      if (lane == 0) tile_flags[kDequantWarps * ts + w] = (unsigned char)flags;
      if (bad != 0) nan_rope(smem_u32(slot) + kRopeOff + (uint32_t)(kDequantRows * w) * 64, bad);
      fence_proxy_async_smem();  // the tensor core reads the tile through the async proxy
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kTFull + ts]);
      if (++m == (uint32_t)nraw) {
        m = 0;
        mphase ^= 1;
      }
      if (++ts == (uint32_t)nts) {
        ts = 0;
        tphase ^= 1;
      }
    }
    // Drain: every slot's last release (a tensor-core commit) lands before the
    // CTA may retire.  Bounded; skipped after an abort.
    if (ok && w == 0) {
      for (uint32_t q = 0; q < (uint32_t)nts && q < ntiles; ++q) {
        const uint32_t last = q + ((ntiles - 1 - q) / nts) * nts;  // last tile in slot q
        if (!all_wait(&bars[kTEmpty + q], (last / nts) & 1, abort_s)) break;
      }
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------------ QK issuer
    if (lo < hi) {
      const uint32_t idesc_qk = idesc_bf16_f32(128, kTile, 0, 0);
      const uint64_t kdesc0 = sw128_desc(smem_u32(ring), 16, 1024);
      const uint64_t qrdesc0 = sw64_desc(smem_u32(qr_s), 512);
      const uint64_t rdesc0 = sw64_desc(smem_u32(ring + kRopeOff), 512);
      uint32_t ts = 0, tphase = 0;
      SegIter it;
      it.init(a.tile_start, U, lo, hi);
      int32_t u, t0, nt, ks;
      bool wh;
      uint32_t j = 0;
      int seg = 0;
      bool ok = true;
      while (ok && it.next(&u, &t0, &nt, &wh, &ks)) {
        // the query's rope dims, once the previous segment's products have read the last ones
        if (!all_wait(&bars[kQEmpty], (seg & 1) ^ 1, abort_s)) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&bars[kQFull], Rg * 64);
          tma_load_2d(qr_s, &tmap_q64, &bars[kQFull], 2 * kOwnChunks * kChunkDims + kRopeHalf * (int)rank,
                      u / a.n_held * a.R_total + g * Rg);
        }
#pragma unroll 1
        for (int jj = 0; jj < nt; ++jj, ++j) {
          if (!all_wait(&bars[kTFull + ts], tphase, abort_s) ||
              (jj == 0 && !all_wait(&bars[kQFull], seg & 1, abort_s)) ||
              (j >= 1 && !all_wait(&bars[kSFree], (j - 1) & 1, abort_s))) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (elect_one()) {
            const uint32_t d = tmem + kSCol;
            const uint32_t soff = (ts * kSlotBytes) >> 4;
            const uint64_t kd = kdesc0 + soff;
#pragma unroll
            for (int i = 0; i < kOwnChunks; ++i)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_bf16_ts(d, tmem + kQCol + 32 * i + 8 * kk, kd + i * (kChunkBytes >> 4) + 2 * kk, idesc_qk,
                            (i | kk) != 0);
#pragma unroll
            for (int kk = 0; kk < kRopeHalf / 16; ++kk)
              mma_bf16_ss(d, qrdesc0 + 2 * kk, rdesc0 + soff + 2 * kk, idesc_qk, 1);
            mma_commit(&bars[kSFull]);
            if (jj == nt - 1) mma_commit(&bars[kQEmpty]);
          }
          __syncwarp();
          if (++ts == (uint32_t)nts) {
            ts = 0;
            tphase ^= 1;
          }
        }
        ++seg;
      }
    }
  } else if (warp == kPvWarp) {
    // ------------------------------------------------------------------ PV issuer
    if (lo < hi) {
      const uint32_t idesc_pv = idesc_bf16_f32(128, 256, 0, 1);
      const uint64_t vdesc0 = sw128_desc(smem_u32(ring), kChunkBytes, 1024);
      SegIter it;
      it.init(a.tile_start, U, lo, hi);
      int32_t u, t0, nt, ks;
      bool wh;
      uint32_t j = 0, ts = 0, tphase = 0;
      int seg = 0;
      bool ok = true;
      while (ok && it.next(&u, &t0, &nt, &wh, &ks)) {
#pragma unroll 1
        for (int jj = 0; jj < nt; ++jj, ++j) {
          // the tile's flags; P(j) ready; the first product of a segment also needs the
          // previous segment's O read out
          if (!all_wait(&bars[kTFull + ts], tphase, abort_s)) { ok = false; break; }
          const uint32_t flags = *reinterpret_cast<const volatile uint32_t*>(tile_flags + kDequantWarps * ts);
          if (!all_wait(&bars[kPFull + (j & 1)], (j >> 1) & 1, abort_s) ||
              (jj == 0 && seg >= 1 && !all_wait(&bars[kOFree], (seg - 1) & 1, abort_s))) {
            ok = false;
            break;
          }
          if (flags & 0x04040404u) zero_nan_values(smem_u32(ring) + ts * kSlotBytes);
          tc_fence_after();
          if (elect_one()) {
            const uint32_t pa = tmem + kPCol + 32 * (j & 1);  // P(j): 64 bf16 = 32 columns
            const uint64_t vd = vdesc0 + ((ts * kSlotBytes) >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_bf16_ts(tmem + kOCol, pa + 8 * kk, vd + kk * (2048 >> 4), idesc_pv, !(jj == 0 && kk == 0));
            mma_commit(&bars[kTEmpty + ts]);
            mma_commit(&bars[kPVDone + (j & 1)]);
          }
          __syncwarp();
          if (++ts == (uint32_t)nts) {
            ts = 0;
            tphase ^= 1;
          }
        }
        ++seg;
      }
    }
  } else if (warp < kSoftmaxWarps && 32 * (warp & 3) + kHalfRows * (warp >> 2) < Rg) {
    // ------------------------------------------------------------------ score exchange, softmax, epilogue
    // Warp w < 8 serves the 16 rows [r0, r0 + 16), r0 = 32 (w % 4) + 16 (w / 4), of
    // every tile, with two threads per row: thread t takes row r0 + t % 16.  This CTA
    // runs the softmax of keys [32 r, 32 r + 32); thread t has the 16 of them from
    // 16 (t / 16) on (and O columns [128 (t / 16), +128)).  Per tile j:
    //   ship S(j): the partial scores of the peer's 32 keys, staged in buffer j & 1 and
    //     sent with one bulk copy; those of the own keys stay in registers;
    //   wait for the peer's S(j), add, ship S(j + 1);
    //   take in the peer's P(j - 1), release PV(j - 1);
    //   softmax of the own keys, P(j) to TMEM and, with its row references and sums, to
    //     the peer.
    // So both messages travel during other work.  A message of tile j is staged in
    // buffer j & 1 and lands in the peer's buffer (j & 1) ^ 1: it is staged where the
    // peer's message of tile j - 1 has just been read, and lands where the peer staged
    // its own of tile j - 1, which has arrived here.  Both conditions are local, so no
    // barrier guards the buffers.
    //   The CTAs need not agree on a row's reference m (P = 2^(s - m)): references are
    // whole numbers, so the peer's P is brought to this CTA's by a power of two, exactly.
    // Each CTA raises its own when the own scores, or the peer's reference, pass it by
    // more than 8, and scales its half of O, P and the sum by a power of two.
    // Waits are warp-wide and bounded, so a timeout drains every thread.
    const int r0 = 32 * (warp & 3) + kHalfRows * (warp >> 2);
    const int ch = warp;  // exchange channel
    const int h = lane >> 4;
    const int row = r0 + (lane & 15);
    const uint32_t lane_addr = (uint32_t)r0 << 16;
    if (lo < hi) {
      auto wwait = [&](uint64_t* bar, uint32_t parity) -> bool { return warp_wait(bar, parity, abort_s, lane); };
      auto wland = [&](uint64_t* bar, uint32_t parity) -> bool { return warp_wait_cluster(bar, parity, abort_s, lane); };
      const uint32_t peer = rank ^ 1u;
      const uint32_t s_own = smem_u32(smem) + sl.s + (uint32_t)(r0 / kHalfRows) * kSWarpBytes;  // this warp's parts
      const uint32_t p_own = smem_u32(smem) + sl.p + (uint32_t)(r0 / kHalfRows) * kPWarpBytes;
      const uint32_t s_peer = mapa_shared(s_own, peer), p_peer = mapa_shared(p_own, peer);
      uint64_t* const s_land = &bars[kSLand + ch];
      uint64_t* const p_land = &bars[kPLand + ch];
      const uint32_t s_land_peer = mapa_shared(smem_u32(s_land), peer), p_land_peer = mapa_shared(smem_u32(p_land), peer);
      uint32_t own[16];  // partial scores of the own keys of the tile shipped last
      // ships the partial scores of the tile of parity `odd`: staged at s_own + odd * sbuf
      auto ship_s = [&](uint32_t odd) -> bool {
        if (!wwait(&bars[kSFull], odd)) return false;
        tc_fence_after();
        uint32_t oth[16];
        tmem_ld16x2_16_pair_sync<16>(tmem + lane_addr + kSCol + kOwnKeys * rank, own,
                                     tmem + lane_addr + kSCol + kOwnKeys * (rank ^ 1u), oth);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kSFree]);
        const uint32_t to = odd ? sl.sbuf : 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          st_shared_v4(s_own + to + lane * 16 + 512 * i, oth[4 * i], oth[4 * i + 1], oth[4 * i + 2], oth[4 * i + 3]);
        fence_proxy_async_smem();  // the copy engine reads what the warp staged
        __syncwarp();
        if (lane == 0)
          bulk_copy_to_peer(s_peer + sl.sbuf - to, s_own + to, kSWarpBytes, s_land_peer + 64 * (odd ^ 1u));
        return true;
      };
      float m_ref = kNoRef;     // the row's reference (log2 units, a whole number)
      float l = 0.f;            // this thread's part of the row's running sum
      // takes in the peer's P of tile jp, the segment's `first` or a later one, and releases PV(jp)
      auto take_p = [&](uint32_t jp, bool first) -> bool {
        const uint32_t odd = jp & 1;
        uint64_t* const land = p_land + 8 * (odd ^ 1u);
        if (!wland(land, (jp >> 1) & 1)) return false;
        const uint32_t src = p_own + (odd ? 0u : sl.pbuf);
        uint32_t pp[8];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint4 w4 = ld_shared_v4(src + 512 * i + lane * 16);
          pp[4 * i] = w4.x; pp[4 * i + 1] = w4.y; pp[4 * i + 2] = w4.z; pp[4 * i + 3] = w4.w;
        }
        const float2 ml = ld_shared_f32x2(src + kPOff + 8 * (lane & 15));  // the peer's reference and row sum
        __syncwarp();  // every lane's reads are done
        if (lane == 0) mbar_arrive_expect_tx(land, kPWarpBytes);
        const uint32_t pc = tmem + lane_addr + kPCol + 32 * odd;
        const bool raise = ml.x > m_ref + (first ? 0.f : kRescaleThreshold);
        if (__any_sync(0xffffffffu, raise)) {
          const float alpha = raise ? pow2(m_ref - ml.x) : 1.f;
          if (!first) {
            if (!wwait(&bars[kPVDone + (odd ^ 1u)], ((jp - 1) >> 1) & 1)) return false;
            tc_fence_after();
            rescale_rows(tmem + lane_addr + kOCol, alpha);
          }
          tmem_st_wait();  // the own P is read back
          uint32_t mine[8];
          tmem_ld16x2_8_sync<8>(pc + 16 * rank, mine);
          scale_bf16x2(mine, alpha);
          tmem_st16x2_8<8>(pc + 16 * rank, mine);
          l *= alpha;
          if (raise) m_ref = ml.x;
        }
        const float f = pow2(ml.x - m_ref);
        scale_bf16x2(pp, f);
        if (h == 0) l = fmaf(ml.y, f, l);
        tmem_st16x2_8<8>(pc + 16 * (rank ^ 1u), pp);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kPFull + odd]);
        return true;
      };
      SegIter it;
      it.init(a.tile_start, U, lo, hi);
      int32_t u, t0, nt, kslot;
      bool whole;
      uint32_t j = 0;  // tile index within the range
      int seg = 0;
      bool ok = true;
      const int grow = g * Rg + row;
      const bool has_row = row < Rg && grow < a.R_total;
      // This warp's rows of the query chunks 4r .. 4r + 3 of request bq into TMEM for
      // segment sq, once QK of segment sq - 1 no longer reads the last ones.  Loaded
      // 8 lanes to a 128-byte row piece (a row per lane touches 32 lines a load, and
      // took 3 us), and turned to a row per thread through the part of the score
      // buffers that the next tile is staged in.
      const int q_row = lane >> 3, q_piece = lane & 7;
      auto q_src = [&](int bq, int i) {  // of row 4 i + lane / 8
        return a.q + ((int64_t)bq * a.R_total + g * Rg + r0 + 4 * i + q_row) * kDk + 256 * (int)rank + 8 * q_piece;
      };
      auto q_has = [&](int i) {
        const int rr = r0 + 4 * i + q_row;
        return rr < Rg && g * Rg + rr < a.R_total;
      };
      auto load_q = [&](int bq, int sq, uint32_t turn) -> bool {
        uint4 qv[4][4];
#pragma unroll
        for (int c = 0; c < kOwnChunks; ++c)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            qv[c][i] = q_has(i) ? __ldg(reinterpret_cast<const uint4*>(q_src(bq, i) + kChunkDims * c))
                                : make_uint4(0, 0, 0, 0);
        if (!wwait(&bars[kQEmpty], (sq & 1) ^ 1)) return false;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < kOwnChunks; ++c) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int rr = 4 * i + q_row;
            st_shared_v4(turn + rr * 128 + ((uint32_t)(q_piece ^ (rr & 7)) << 4), qv[c][i].x, qv[c][i].y, qv[c][i].z,
                         qv[c][i].w);
          }
          __syncwarp();
          uint32_t r[16];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint4 w4 = ld_shared_v4(turn + (lane & 15) * 128 + ((uint32_t)((4 * h + k) ^ (lane & 7)) << 4));
            r[4 * k] = w4.x; r[4 * k + 1] = w4.y; r[4 * k + 2] = w4.z; r[4 * k + 3] = w4.w;
          }
          tmem_st16x2_16<16>(tmem + lane_addr + kQCol + 32 * c, r);
          __syncwarp();
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kQFull]);
        return true;
      };
      const int t_row = has_row ? grow / a.H + 1 : 0;  // visible positions beyond S - q_len
      // Each segment's description and length come from the segment before it
      // (peeked and loaded there), so a segment start waits on no global load.
      bool have = it.next(&u, &t0, &nt, &whole, &kslot);
      int64_t S_cur = 0;
      if (have) {
        S_cur = a.seq_lens[u / a.n_held];
        ok = load_q(u / a.n_held, 0, s_own);
      }
      while (ok && have) {
        const int b = u / a.n_held, rs = u % a.n_held;
        ++seg;
        SegIter nx = it;
        int32_t u2 = 0, t02 = 0, nt2 = 0, ks2 = 0;
        bool wh2 = false, has_next = false;
        int64_t S_next = 0;
        const int64_t S = S_cur;
        // this thread's keys k < lim of a tile are visible; lim for tile t0 - 1, in 32
        // bits (a shard's rows of a request are fewer than 2^31)
        int32_t lim = 0;
        if (S >= a.q_len) {
          const int64_t n = rows_below(a, rs, S - a.q_len + t_row);
          lim = has_row ? (int32_t)(n - ((int64_t)t0 - 1) * kTile) - kOwnKeys * (int)rank - 16 * h : 0;
        }
        m_ref = kNoRef;
        l = 0.f;
        // Step jj works on tile j = jj of the segment; steps -1 and nt only ship the
        // first tile and take in the last, so that each part is in the code once.
        const uint32_t j0 = j;
#pragma unroll 1
        for (int jj = -1; jj <= nt; ++jj) {
          const bool tile = jj >= 0 && jj < nt;
          j = j0 + (uint32_t)jj;
          const uint32_t odd = j & 1;
          uint32_t s[16];
          if (tile) {
            // ---- scores of the own keys: this CTA's partial scores + the peer's
            uint64_t* const land = s_land + 8 * (odd ^ 1u);
            if (!wland(land, (j >> 1) & 1)) { ok = false; break; }
            const uint32_t src = s_own + (odd ? 0u : sl.sbuf) + lane * 16;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint4 far = ld_shared_v4(src + 512 * i);
              f2_unpack(f2_add(f2_pack(own[4 * i], own[4 * i + 1]), f2_pack(far.x, far.y)), s[4 * i], s[4 * i + 1]);
              f2_unpack(f2_add(f2_pack(own[4 * i + 2], own[4 * i + 3]), f2_pack(far.z, far.w)), s[4 * i + 2],
                        s[4 * i + 3]);
            }
            __syncwarp();  // every lane's reads are done
            if (lane == 0) mbar_arrive_expect_tx(land, kSWarpBytes);
          }
          if (jj + 1 < nt && !ship_s(odd ^ 1u)) { ok = false; break; }
          if (jj > 0 && !take_p(j - 1, jj == 1)) { ok = false; break; }
          if (!tile) continue;
          // ---- online softmax of the own keys of tile j
          lim -= kTile;
          if (lim < 16) {
#pragma unroll
            for (int k = 0; k < 16; ++k)
              if (k >= lim) s[k] = __float_as_uint(-INFINITY);
          }
          float mx = fmax_nan(__uint_as_float(s[0]), __uint_as_float(s[1]));
          float my = fmax_nan(__uint_as_float(s[2]), __uint_as_float(s[3]));
#pragma unroll
          for (int k = 4; k < 16; k += 4) {
            mx = fmax3_nan(mx, __uint_as_float(s[k]), __uint_as_float(s[k + 1]));
            my = fmax3_nan(my, __uint_as_float(s[k + 2]), __uint_as_float(s[k + 3]));
          }
          mx = fmax_nan(mx, my);
          mx = fmax_nan(mx, __shfl_xor_sync(0xffffffffu, mx, 16));  // the row's other 16 keys
          float mt = mx * a.scale_log2;  // scale > 0: the max commutes with the scaling
          bool raise = !(mt <= m_ref + kRescaleThreshold);  // also the row's first visible key, and NaN
          if (__any_sync(0xffffffffu, raise)) {
            if (__any_sync(0xffffffffu, mx != mx)) {
              // Keys on a bad page leave the softmax; the maximum is that of the rest, without
              // the NaN that the cache or the query holds.  (8 keys at a time, swapping the
              // halves: the tile loop that this sits in pays for its length, 2296 us against
              // 2316 for 64 requests of 128k tokens.)
              uint32_t bad = bad_groups(&bars[kTFull], tile_flags + 2 * rank + h, j, nts, abort_s);
              if (bad == ~0u) { ok = false; break; }
              mx = -INFINITY;
#pragma unroll 1
              for (int half = 0; half < 2; ++half, bad >>= 1) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  if (bad & 1) s[k] = __float_as_uint(-INFINITY);
                  mx = fmaxf(mx, __uint_as_float(s[k]));
                  const uint32_t x = s[k];
                  s[k] = s[k + 8];
                  s[k + 8] = x;
                }
              }
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
              mt = mx * a.scale_log2;
              raise = mt > m_ref + kRescaleThreshold;
            }
            float alpha = 1.f;
            if (raise) {
              const float m_new = ceilf(mt);
              alpha = pow2(m_ref - m_new);  // 0 without a reference yet: O and l are 0 too
              m_ref = m_new;
            }
            if (jj > 0) {  // O holds something: scale it once PV(j - 1) is done
              if (!wwait(&bars[kPVDone + (odd ^ 1u)], ((j - 1) >> 1) & 1)) { ok = false; break; }
              tc_fence_after();
              rescale_rows(tmem + lane_addr + kOCol, alpha);
            }
            l *= alpha;
          }
          const float cs = a.scale_log2;
          const uint64_t cs2 = f2_pack(__float_as_uint(cs), __float_as_uint(cs));
          const uint64_t nm2 = f2_pack(__float_as_uint(-m_ref), __float_as_uint(-m_ref));
          uint64_t ps[2] = {0, 0};  // pairs of partial row sums (+0.f bits)
          uint32_t pk[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            uint32_t x0, x1;
            f2_unpack(f2_fma(f2_pack(s[2 * k], s[2 * k + 1]), cs2, nm2), x0, x1);
            const float p0 = fast_exp2(__uint_as_float(x0));
            const float p1 = fast_exp2(__uint_as_float(x1));
            ps[k & 1] = f2_add(ps[k & 1], f2_pack(__float_as_uint(p0), __float_as_uint(p1)));
            __nv_bfloat162 hh = __floats2bfloat162_rn(p0, p1);
            pk[k] = *reinterpret_cast<uint32_t*>(&hh);
          }
          float sum;
          {
            uint32_t a0, a1;
            f2_unpack(f2_add(ps[0], ps[1]), a0, a1);
            sum = __uint_as_float(a0) + __uint_as_float(a1);
          }
          l += sum;
          sum += __shfl_xor_sync(0xffffffffu, sum, 16);
          // ---- P(j): to the peer, and to TMEM (the A operand of the PV product) once
          // PV(j - 2) has read the buffer
          {
            const uint32_t to = odd ? sl.pbuf : 0u;
#pragma unroll
            for (int i = 0; i < 2; ++i)
              st_shared_v4(p_own + to + 512 * i + lane * 16, pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
            if (h == 0) st_shared_f32x2(p_own + to + kPOff + 8 * lane, m_ref, sum);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
              bulk_copy_to_peer(p_peer + sl.pbuf - to, p_own + to, kPWarpBytes, p_land_peer + 64 * (odd ^ 1u));
          }
          if (j >= 2 && !wwait(&bars[kPVDone + odd], ((j - 2) >> 1) & 1)) { ok = false; break; }
          tc_fence_after();
          tmem_st16x2_8<8>(tmem + lane_addr + kPCol + 32 * odd + 16 * rank, pk);  // complete before take_p releases it
          if (jj == 0) {
            has_next = nx.next(&u2, &t02, &nt2, &wh2, &ks2);
            if (has_next) {
              S_next = a.seq_lens[u2 / a.n_held];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (q_has(i) && q_piece < kOwnChunks)
                  asm volatile("prefetch.global.L2 [%0];" ::"l"(q_src(u2 / a.n_held, i) + 56 * q_piece));
            }
          }
        }
        if (!ok) break;
        j = j0 + (uint32_t)nt;
        // (j is the next tile: it is staged at s_own + (j & 1) * sbuf)
        if (has_next && !load_q(u2 / a.n_held, seg, s_own + ((j & 1) ? sl.sbuf : 0u))) { ok = false; break; }
        const float l_row = l + __shfl_xor_sync(0xffffffffu, l, 16);
        // ---------------- epilogue: O rows / l -> o (this CTA's 256 dims), lse
        const uint32_t jl = j - 1;
        if (!wwait(&bars[kPVDone + (jl & 1)], (jl >> 1) & 1)) { ok = false; break; }
        tc_fence_after();
        const int rows_here = min(Rg, a.R_total - g * Rg);
        const bool writes = row < rows_here;
        const int64_t out_base = ((int64_t)rs * a.B + b) * a.R_total + g * Rg;
        const int64_t piece_base = (int64_t)(2 * v + kslot) * a.R_total + g * Rg;
        const float inv = l_row != 0.f ? 1.f / l_row : 0.f;  // 0: no key seen; a NaN stays one
        // staging for the output rows: this warp's part of the buffer the last tile's
        // peer scores were read from
        store_rows_q4(a, tmem + lane_addr + kOCol, rows_here, whole, out_base, piece_base, r0, 256 * (int)rank + 128 * h,
                      inv, s_own + ((jl & 1) ? 0u : sl.sbuf));
        if (writes && h == 0 && rank == 0) {
          const float lse2 = l_row != 0.f ? m_ref + log2f(l_row) : -INFINITY;
          if (whole)
            a.lse_part[out_base + row] = a.base2 ? lse2 : lse2 * kLn2;
          else
            a.piece_lse[piece_base + row] = lse2;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kOFree]);
        it = nx;  // the segment just peeked (its fields below)
        have = has_next;
        u = u2, t0 = t02, nt = nt2, whole = wh2, kslot = ks2;
        S_cur = S_next;
      }
    }
  } else if (warp < kSoftmaxWarps) {
    // No rows of the group: zero this warp's 16 TMEM lanes of the P and query
    // columns once, so the M = 128 products carry zeros in the padding rows (their
    // query rope rows are zero too; less power).
    const uint32_t zl = (uint32_t)(32 * (warp & 3) + kHalfRows * (warp >> 2)) << 16;
    uint32_t z[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) z[i] = 0u;
    tmem_st16x2<32>(tmem + zl + kPCol, z);
    tmem_st16x2<32>(tmem + zl + kQCol, z);
    tmem_st16x2<32>(tmem + zl + kQCol + 64, z);
    tmem_st_wait();
  }

  if (*abort_s && tid == 0) flag(a.status, DCP_STATUS_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  // The peer may still have stores or arrivals addressed to this CTA's shared
  // memory; retire the pair together.  After an abort, allow in-flight tensor
  // core commits (microseconds) to land first.
  if (*abort_s) __nanosleep(100000);
  cluster_sync();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

}  // namespace

#include "dcp_decode_q4_few.cuh"

namespace {

// ---------------------------------------------------------------------------- host side
SmemLimit g_few_smem;
PairKernel g_kernel(reinterpret_cast<const void*>(&partial_q4_kernel), kThreads);

// Whether a call takes the few-row kernel (its header has both sides' times).
bool few_rows(int q_len, int H) { return q_len * H <= kFewRows; }

bool make_plan(const dcp_layout_t* layout, int n_held, int B, int q_len, int H, Plan* p) {
  plan_groups(q_len, H, p);
  if (few_rows(q_len, H)) {
    const int sms = sm_count_current();
    if (sms <= 0) return false;
    p->nts = 0;
    p->V = 2 * sms;  // two CTAs an SM
    p->smem = sizeof(FewSmem);
    plan_workspace(layout, n_held, B, q_len * H, p);
    return true;
  }
  p->nts = kMaxSlots;
  p->nraw = (int)((kSmemBudget - smem_layout(p->Rg, p->nts, 0).total) / kRawBytes);
  if (p->nraw > kMaxRaw) p->nraw = kMaxRaw;
  p->smem = smem_layout(p->Rg, p->nts, p->nraw).total;
  return p->nraw >= 1 && plan_ranges(layout, n_held, B, q_len, H, g_kernel, p);
}

// Part [offset, offset + inner elements) of every 416-byte row, as boxes of
// [box_rows][box_inner elements].
bool make_tmap_q4(CUtensorMap* m, CUtensorMapDataType type, CUtensorMapSwizzle swizzle, const void* arena, int offset,
                  int inner, uint64_t rows, uint32_t box_inner, uint32_t box_rows) {
  auto enc = tmap_encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)kQ4RowBytes};
  cuuint32_t box[2] = {box_inner, box_rows};
  cuuint32_t es[2] = {1, 1};
  void* base = const_cast<unsigned char*>(static_cast<const unsigned char*>(arena)) + offset;
  return enc(m, type, 2, base, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
             CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

extern "C" size_t dcp_mla_decode_workspace_size_q4(const dcp_layout_t* layout, int32_t shard_begin,
                                                   int32_t shard_end, int32_t B, int32_t q_len, int32_t H) {
  Plan p;
  if (!size_args_ok(layout, shard_begin, shard_end, B, q_len, H) ||
      !make_plan(layout, shard_end - shard_begin, B, q_len, H, &p))
    return 0;
  return p.ws_total;
}

extern "C" int32_t dcp_mla_decode_partial_q4(const dcp_layout_t* layout, int32_t shard_begin, int32_t shard_end,
                                             const void* q, int32_t B, int32_t q_len, int32_t H,
                                             const void* arena, int64_t pool_pages,
                                             const int32_t* block_table, int64_t bt_stride, int64_t max_pages,
                                             const int64_t* seq_lens, float scale, int32_t lse_base,
                                             void* o_part, int32_t o_part_dtype, float* lse_part,
                                             void* workspace, size_t workspace_bytes,
                                             int32_t* status, void* stream) {
  const DecodeCall c{layout, shard_begin, shard_end, q, B, q_len, H, arena, pool_pages, block_table, bt_stride,
                     max_pages, seq_lens, scale, lse_base, o_part, o_part_dtype, lse_part, status, stream};
  int32_t rc = check_decode_args(c);
  if (rc != DCP_OK) return rc;
  Plan p;
  if (!make_plan(layout, shard_end - shard_begin, B, q_len, H, &p)) return DCP_ERR_CUDA;
  rc = check_workspace(p, workspace, workspace_bytes);
  if (rc != DCP_OK) return rc;
  const TcArgs a = device_args(p, c, workspace);
  if (few_rows(q_len, H)) {
    if (!g_few_smem.ensure(reinterpret_cast<const void*>(&few_q4_kernel), p.smem)) return DCP_ERR_CUDA;
    return launch_decode(p, a, kFewThreads, stream, [&](cudaLaunchConfig_t lc) {
      lc.gridDim = dim3((unsigned)p.V);
      return cudaLaunchKernelEx(&lc, few_q4_kernel, static_cast<const unsigned char*>(arena), a);
    });
  }
  const uint64_t rows = (uint64_t)a.n_held * a.pool_rows;
  const uint32_t box = (uint32_t)p.box_rows;
  CUtensorMap tq64, tcode, tscale, trope;
  if (!make_tmap(&tq64, q, (uint64_t)B * a.R_total, (uint32_t)p.Rg, true)) return DCP_ERR_CUDA;
  if (!make_tmap_q4(&tcode, CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_128B, arena, 0, kQ4ScaleOff, rows, 128,
                    box) ||
      !make_tmap_q4(&tscale, CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_NONE, arena, kQ4ScaleOff,
                    kDv / kQ4Group, rows, 16, box) ||
      !make_tmap_q4(&trope, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, CU_TENSOR_MAP_SWIZZLE_64B, arena, kQ4RopeOff, kDk - kDv,
                    rows, kRopeHalf, box))
    return DCP_ERR_CUDA;
  if (!g_kernel.ensure_smem(p.smem)) return DCP_ERR_CUDA;
  return launch_decode(p, a, kThreads, stream, [&](const cudaLaunchConfig_t& lc) {
    return cudaLaunchKernelEx(&lc, partial_q4_kernel, tq64, tcode, tscale, trope, static_cast<const unsigned char*>(arena), a);
  });
}
