// dcp_decode.cu — per-shard partial attention (o_r, lse_r) for absorbed MLA on sm_103a.
//
// Sources: "MLA 的 Decode Context Parallelism", section 2 (absorbed form: one
// 576-d KV head shared by all query heads; values are the first 512 dims) and
// section 3 (each rank returns its locally normalised output and its LSE);
// "Decode Context Parallelism" (zdszero), "Core abstraction" idea 2 and
// "Theory" (the (Z, N) merge operator: a shard may itself be split into pieces
// that are merged the same way); SGLang "Decode context parallelism",
// "DCP x speculative decoding" (causal mask in global positions, from the shard
// rank and the global lengths).
//
// Design: persistent 2-CTA clusters, one CTA per SM, 384 threads each:
//   warps 0-7   softmax and score exchange: warp w serves 16 query rows
//               (two threads per row, 32 keys each); it loads its rows of this
//               CTA's query chunks into TMEM once per segment, ships its rows
//               of each partial score tile to the peer, runs the online
//               softmax and writes its rows of O at a segment end.
//   warp 9      PV issuer (one thread).
//   warp 10     TMA producer: this CTA's share of every KV tile (64 local rows)
//               into a ring of tile slots, an L2 prefetch two tiles ahead, and
//               the query's shared-memory operands once per segment.  The warp
//               fetches block-table entries 32 tiles at a time.
//   warp 11     QK issuer (one thread) and TMEM owner.
// A cluster handles a group of at most 128 query rows.  The 576 key dims are
// split between the two CTAs: CTA r loads value chunks 4r .. 4r + 3 (dims
// [256 r, 256 r + 256), one 3-D box of four 128-byte-swizzled 64 x 64 tiles)
// and rope dims [512 + 32 r, 512 + 32 r + 32) (64-byte swizzle).  Per tile j,
// in each CTA:
//   S_j^r = Q[:, K_r] K_j[:, K_r]^T   M=128 rows, N=64 KV rows, K=288: query
//                                     chunks 4r, 4r+1 from TMEM, chunks 4r+2,
//                                     4r+3 and the rope half from shared
//                                     memory -> TMEM fp32
//   each softmax warp stages its rows of S_j^r in shared memory and one bulk
//   copy ships them to the peer (credited on the peer's mbarrier; two buffers
//   per CTA swap the staging and receiving roles every tile); each CTA forms
//   S_j = S_j^0 + S_j^1 (fp32 addition is commutative, so both CTAs hold the
//   same bits and take the same softmax decisions);
//   P_j   = exp2(S_j*scale*log2e - m)  online softmax with lazy rescaling,
//                                     bf16 pairs in their own TMEM columns
//   O_r  += P_j V_j[:, dims of r]     M=128 rows (A = P from TMEM), N=256,
//                                     K=64 KV rows                   -> TMEM fp32
// Each KV byte crosses HBM once and reaches one SM's shared memory once; the
// tile's chunks stay in the ring from the QK product to the PV product (V = the
// first 512 dims of the same rows).  TMEM per CTA: O (256 columns), two S
// tiles (2 x 64), two P tiles (2 x 32) and two query chunks (64).  An S tile
// is free as soon as every softmax warp has read it, so QK products run up to
// two tiles ahead of the softmax while the exchange is in flight.
//
// The work split over clusters, its planner and the merge of cut units are in
// dcp_decode.cuh.
#include "dcp_decode.cuh"

namespace {

constexpr int kMaxTileSlots = 8;
constexpr int kL2Ahead = 2;                   // tiles between a tile's L2 prefetch and its ring load
constexpr int kFixedBarSlots = 32;            // mbarriers other than the per-slot ones
constexpr int kThreads = 384;                 // 12 warps (roles below)
// Warp roles.  Warp w runs on SM sub-partition w % 4 and reaches TMEM lanes
// [32 (w % 4), 32 (w % 4) + 32): the softmax and sender warps of row quarter q
// are q and 4 + q.  The tensor-core issuer (a polling thread) sits with the
// warps of quarter 3, the quarter a group of up to 96 rows leaves empty, and
// the producer with quarter 2; warps 8 and 9 have no role.
constexpr int kProducerWarp = 10;
constexpr int kMmaWarp = 11;                  // QK issuer and TMEM owner
constexpr int kPvWarp = 9;                    // PV issuer
constexpr uint32_t kOCol = 0;                 // TMEM columns [0, 256): O, rows on lanes
constexpr uint32_t kSCol = 256;               // [256, 384): two S tiles of 64 fp32 columns
constexpr uint32_t kPCol = 384;               // [384, 448): P of two tiles as bf16 pairs (2 x 32)
constexpr uint32_t kQCol = 448;               // [448, 512): query chunks 4r, 4r + 1 as bf16 pairs
constexpr int kQTmemChunks = 2;               // query chunks 4r + 2, 4r + 3 are read from shared memory

struct SmemLayout {
  uint32_t qc, qr, x, xbuf, ring, rope, bars, misc, total;
};

__host__ __device__ inline SmemLayout smem_layout(int Rg, int nts) {
  SmemLayout s;
  // The M = 128 shared-memory A operands hold the group's Rg rows; the products
  // also read the 128 - Rg rows that follow into TMEM lanes no thread reads
  // back.  Query chunk 4r + 2 is given all 128 rows, zeroed, so its padding
  // rows multiply zeros (less power at the power cap); chunk 4r + 3 and the
  // rope dims are followed by other data, as the ring needs the space.
  s.qc = 0;                                        // query chunks 4r + 2 ([128][64], rows >= Rg zero), 4r + 3 ([Rg][64]), bf16, 128-byte swizzle
  s.qr = (128 + (uint32_t)Rg) * 128;               // query rope dims [32r, 32r + 32): [Rg][32], 64-byte swizzle
  s.x = round1024(s.qr + (uint32_t)Rg * 64);       // two [Rg][64] fp32 buffers: partial scores staged / received
  s.xbuf = round1024((uint32_t)Rg * kXRowBytes);
  s.ring = s.x + 2 * s.xbuf;                       // tile slots: 4 value chunks + this CTA's rope half
  s.rope = s.ring;                                 // (kept for the layout struct; rope lives in the slots)
  s.bars = s.ring + nts * kSlotBytes;
  s.misc = s.bars + (kFixedBarSlots + 2 * kMaxTileSlots) * 8;
  s.total = s.misc + 64;
  return s;
}

enum Bar { kQFull = 0, kQEmpty, kSFull0, kSFull1, kSFree0, kSFree1, kPFull0, kPFull1, kPVDone0, kPVDone1, kOFree,
           kXFull = 11,  // [2 buffers][8 channels]: the peer's partial scores of a channel's rows have landed
           kNumFixedBars = 27 };
static_assert(kNumFixedBars <= kFixedBarSlots, "fixed barriers");

// ---------------------------------------------------------------------------- main kernel
// A 2-CTA cluster per (work range, row group).  CTA `rank` loads key/value dims
// [256 rank, 256 rank + 256) and 32 rope dims of every tile,
// computes its partial scores over them, swaps partial scores with its peer and
// accumulates its own 256 value dims of O.  Both CTAs walk the same tile
// sequence; the score exchange is double-buffered and S tiles are released as
// soon as they have been read, so QK products run up to two tiles ahead of the
// softmax while the exchange is in flight.
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    partial_tc_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_kv,
                      const __grid_constant__ CUtensorMap tmap_q64, const __grid_constant__ CUtensorMap tmap_kv64,
                      const __grid_constant__ CUtensorMap tmap_kv4, TcArgs a) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  // The layout needs a 1024-byte aligned base and the launch reserves no slack
  // for aligning it here: every CTA of the launch sees the same base, so a
  // misaligned one makes all of them stop at once, before any barrier.
  if ((smem_u32(smem_raw) & 1023u) != 0) {
    if (threadIdx.x == 0) flag(a.status, DCP_STATUS_INTERNAL);
    return;
  }
  // launched as a programmatic dependent of the plan kernel: nothing it wrote
  // (the tile prefix sums, the empty units' rows) is read before this
  griddep_wait();
  unsigned char* smem = smem_raw;
  const SmemLayout sl = smem_layout(a.Rg, a.nts);
  unsigned char* qc_s = smem + sl.qc;
  unsigned char* qr_s = smem + sl.qr;
  unsigned char* x_s = smem + sl.x;
  unsigned char* ring = smem + sl.ring;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + sl.bars);
  uint64_t* tfull = bars + kFixedBarSlots;      // tile slot landed
  uint64_t* tempty = tfull + kMaxTileSlots;     // tile slot released by its PV product
  uint32_t* tmem_base_s = reinterpret_cast<uint32_t*>(smem + sl.misc);
  volatile int* abort_s = reinterpret_cast<volatile int*>(smem + sl.misc + 4);

  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  const int cid = blockIdx.x >> 1;  // cluster index
  const int v = cid / a.ngroups;
  const int g = cid % a.ngroups;
  const int Rg = a.Rg;
  const int nts = a.nts;
  int nhalf = 0;  // softmax warps with rows of the group (warp w < 8 serves rows 32 (w % 4) + 16 (w / 4) + [0, 16))
  for (int w = 0; w < 8; ++w) nhalf += 32 * (w & 3) + kHalfRows * (w >> 2) < Rg;
  const int32_t U = a.B * a.n_held;
  const int64_t T = a.tile_start[U];
  const int64_t lo = range_lo(T, v, a.V), hi = range_lo(T, v + 1, a.V);
  const uint32_t ntiles_cta = (uint32_t)(hi - lo);

  if (tid == 0) {
    *abort_s = 0;
    for (int i = 0; i < kNumFixedBars; ++i) mbar_init(&bars[i], 1);
    mbar_init(&bars[kQFull], nhalf + 1);  // softmax warps + the query-chunk TMA
    mbar_init(&bars[kSFree0], nhalf);     // every softmax warp has read the partial scores
    mbar_init(&bars[kSFree1], nhalf);
    mbar_init(&bars[kPFull0], nhalf);
    mbar_init(&bars[kPFull1], nhalf);
    mbar_init(&bars[kOFree], nhalf);
    // The score exchange runs as one channel per softmax warp (its 16 rows), with
    // one single-arrival "landed" barrier per buffer and channel.
    for (int i = 0; i < nts; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 1);
    }
    fence_barrier_init();
    // tile j's partial scores from the peer land in buffer (j & 1) ^ 1: expect tiles 0 and 1
    for (uint32_t j = 0; j < 2 && j < ntiles_cta; ++j)
      for (int w = 0; w < 8; ++w)
        if (32 * (w & 3) + kHalfRows * (w >> 2) < Rg)
          mbar_arrive_expect_tx(&bars[kXFull + 8 * ((j & 1) ^ 1) + w], kHalfRows * kXRowBytes);
  }
  // rows of a page past a request's length are read with zero weight: start from finite zeros
  for (int i = tid; i < nts * kSlotBytes / 16; i += kThreads) reinterpret_cast<uint4*>(ring)[i] = make_uint4(0, 0, 0, 0);
  // query rows past the group are read by the M = 128 products: zeros
  for (int i = tid; i < (int)(sl.x / 16); i += kThreads) reinterpret_cast<uint4*>(qc_s)[i] = make_uint4(0, 0, 0, 0);
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
    // The whole warp walks the tile sequence: its lanes fetch the block-table
    // entries of 32 tiles at a time (the next 32 are already in flight), lane 0
    // takes each tile's page ids by shuffle, waits for the ring slot and issues
    // the TMA copies.  Waits are lane-0 polls broadcast to the warp.
    if (lo < hi) {
      if (lane == 0) {
        prefetch_tmap(&tmap_q);
        prefetch_tmap(&tmap_kv);
        prefetch_tmap(&tmap_q64);
        prefetch_tmap(&tmap_kv64);
        prefetch_tmap(&tmap_kv4);
      }
      SegIter it;
      it.init(a.tile_start, U, lo, hi);
      int32_t u, t0, nt, kslot;
      bool whole;
      uint32_t j = 0;  // tile index within this CTA's range
      int seg = 0;
      bool ok = true;
      const int nbox = kTile / a.box_rows;
      struct Boxes {
        int32_t y[8];
        uint32_t bytes;
      };
      auto box_y = [](const Boxes& bx, int q) -> int32_t {  // register-resident select (no local memory)
        int32_t y = bx.y[0];
#pragma unroll
        for (int i = 1; i < 8; ++i)
          if (q == i) y = bx.y[i];
        return y;
      };
      // lane l: page ids of the boxes of tile tile0 + l (-2: not needed, -1: past the table)
      auto fetch_batch = [&](int b, int64_t nvis, int32_t tile0, int32_t tile_end, int32_t (&pg)[8]) {
        // (local rows and pool rows fit in 32 bits: the host checks the pool size)
        const int32_t tile = tile0 + lane;
        const int32_t rho0 = tile * kTile;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          pg[q] = -2;
          const int32_t rho = rho0 + q * a.box_rows;
          if (tile < tile_end && q < nbox && rho < nvis) {
            const int32_t pidx = rho / a.L.P;
            pg[q] = pidx >= 0 && pidx < a.max_pages ? __ldg(a.bt + (int64_t)b * a.bt_stride + pidx) : -1;
          }
        }
      };
      // lane l: pool rows of the boxes of tile tile0 + l from their page ids (-1: no box).
      // Which boxes are needed is recomputed here, not read from the -2 marks, so a
      // block-table entry of -2 is reported like any other bad page id.
      auto to_rows = [&](int rs, int32_t tile0, int32_t tile_end, int64_t nvis, const int32_t (&pg)[8],
                         int32_t (&yb)[8]) {
        const int32_t tile = tile0 + lane;
        const int32_t rho0 = tile * kTile;
        const int32_t pool0 = rs * (int32_t)a.pool_rows;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          yb[q] = -1;
          if (!(tile < tile_end && q < nbox && rho0 + q * a.box_rows < nvis)) continue;
          if (pg[q] < 0 || pg[q] >= a.pool_pages) {
            if (rank == 0) flag(a.status, DCP_STATUS_BAD_PAGE_ID);
            continue;
          }
          // a box never crosses a page: its height is min(P, 64) and it starts at a
          // multiple of it, so it starts a page when P <= 64
          const int32_t rho = rho0 + q * a.box_rows;
          const int32_t in_page = a.L.P <= kTile ? 0 : rho % a.L.P;
          yb[q] = pool0 + pg[q] * a.L.P + in_page;
        }
      };
      // the same rows without the bad-page report (the batch is checked again when it is issued)
      auto to_rows_quiet = [&](int rs, int32_t tile0, const int32_t (&pg)[8], int32_t (&yb)[8]) {
        const int32_t rho0 = (tile0 + lane) * kTile;
        const int32_t pool0 = rs * (int32_t)a.pool_rows;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const int32_t rho = rho0 + q * a.box_rows;
          yb[q] = (pg[q] < 0 || pg[q] >= a.pool_pages) ? -1 : pool0 + pg[q] * a.L.P + (a.L.P <= kTile ? 0 : rho % a.L.P);
        }
      };
      auto make_boxes = [&](const int32_t (&y)[8], Boxes& bx) {
        bx.bytes = 0;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          bx.y[q] = y[q];
          if (y[q] >= 0) bx.bytes += a.box_rows * 128;
        }
      };
      // one chunk (all its boxes) into `dst`; exactly as many TMA instructions as
      // boxes (predicated-off copies in an unrolled loop still cost issue time)
      auto issue_chunk = [&](const Boxes& bx, unsigned char* dst, uint64_t* bar, int k) {
        if (nbox == 1) {
          if (bx.y[0] >= 0) tma_load_2d(dst, &tmap_kv, bar, k * kChunkDims, bx.y[0]);
        } else {
          for (int q = 0; q < nbox; ++q) {
            const int32_t y = box_y(bx, q);
            if (y >= 0) tma_load_2d(dst + q * a.box_rows * 128, &tmap_kv, bar, k * kChunkDims, y);
          }
        }
      };
      // this CTA's 32 rope dims of the tile: rows of 64 bytes, 64-byte swizzle
      auto issue_rope = [&](const Boxes& bx, unsigned char* dst, uint64_t* bar) {
        const int32_t x = 2 * kOwnChunks * kChunkDims + kRopeHalf * (int)rank;
        if (nbox == 1) {
          if (bx.y[0] >= 0) tma_load_2d(dst, &tmap_kv64, bar, x, bx.y[0]);
        } else {
          for (int q = 0; q < nbox; ++q) {
            const int32_t y = box_y(bx, q);
            if (y >= 0) tma_load_2d(dst + q * a.box_rows * 64, &tmap_kv64, bar, x, y);
          }
        }
      };
      uint32_t ts = 0, tphase = 0;  // ring slot of tile j and its use parity
      auto load_tile = [&](const Boxes& bx) -> bool {
        if (!warp_wait(&tempty[ts], tphase ^ 1, abort_s, lane)) return false;
        if (lane == 0) {
          mbar_arrive_expect_tx(&tfull[ts], bx.bytes * kOwnChunks + bx.bytes / 2);
          unsigned char* dst = ring + ts * kSlotBytes;
          if (nbox == 1) {
            // all four value chunks of the tile with one 3-D box: [4 chunks][64 rows][128 B]
            if (bx.y[0] >= 0) tma_load_3d(dst, &tmap_kv4, &tfull[ts], 0, bx.y[0], kOwnChunks * (int)rank);
          } else {
            for (int i = 0; i < kOwnChunks; ++i)
              issue_chunk(bx, dst + i * kChunkBytes, &tfull[ts], kOwnChunks * (int)rank + i);
          }
          issue_rope(bx, dst + kRopeOff, &tfull[ts]);
        }
        ++j;
        if (++ts == (uint32_t)nts) {
          ts = 0;
          tphase ^= 1;
        }
        return true;
      };
      // A segment's length and the page ids of its first 32 tiles are loaded
      // during the segment before it, so that a segment start waits on no
      // global load.  The early page ids are read without the length (up to
      // max_pages entries of the row); to_rows applies the length when they are
      // used.
      bool have = it.next(&u, &t0, &nt, &whole, &kslot);
      int32_t pgf[8];       // page ids of the boxes of the segment's first 32 tiles
      int64_t nvis_f = 0;   // and its visible rows
      if (have) {
        bool bad0 = false;
        nvis_f = unit_nvis_max(a, u / a.n_held, u % a.n_held, &bad0);
        fetch_batch(u / a.n_held, INT64_MAX, t0, t0 + nt, pgf);
      }
      while (ok && have) {
        const int b = u / a.n_held, rs = u % a.n_held;
        const int64_t nvis = nvis_f;
        const int32_t t_end = t0 + nt;
        // block-table entries of the next 32 tiles are in flight while the
        // current 32 are issued; each lane turns its tile's entries into TMA rows
        int32_t pgn[8], yc[8], yn = -1;  // yn: next batch's first-box rows (L2 prefetch)
        to_rows(rs, t0, t_end, nvis, pgf, yc);
        fetch_batch(b, nvis, t0 + 32, t_end, pgn);
        // the next segment, peeked once this segment's first tile is issued (the
        // peek waits on the unit table): its length and first page ids are then
        // in flight during this segment
        SegIter nx = it;
        int32_t u2 = 0, t02 = 0, nt2 = 0, ks2 = 0;
        bool wh2 = false, has_next = false;
        int32_t y_next = -1;    // first-box row of the next segment's tile `lane` (L2 prefetch)
        bool next_rows = false;
        // the query's chunk 4r + 3 and its rope dims [32r, 32r + 32) for the SS part of QK
        if (!warp_wait(&bars[kQEmpty], (seg & 1) ^ 1, abort_s, lane)) { ok = false; break; }
        if (lane == 0) {
          const int32_t qy = b * a.R_total + g * Rg;
          mbar_arrive_expect_tx(&bars[kQFull], Rg * (2 * 128 + 64));
          for (int i = kQTmemChunks; i < kOwnChunks; ++i)
            tma_load_2d(qc_s + (i - kQTmemChunks) * 128 * 128, &tmap_q, &bars[kQFull],
                        (kOwnChunks * (int)rank + i) * kChunkDims, qy);
          tma_load_2d(qr_s, &tmap_q64, &bars[kQFull], 2 * kOwnChunks * kChunkDims + kRopeHalf * (int)rank, qy);
        }
        ++seg;
        for (int jj = 0; jj < nt && ok; ++jj) {
          if (jj > 0 && (jj & 31) == 0) {
            to_rows(rs, t0 + jj, t_end, nvis, pgn, yc);
            fetch_batch(b, nvis, t0 + jj + 32, t_end, pgn);
          }
          if (nbox == 1) {
            // The ring holds a few tiles, fewer than HBM latency times the tile
            // rate: each tile is also prefetched into L2 kL2Ahead tiles before its
            // ring load, so that the load finds it there.
            // The next batch's rows, once its block-table entries have arrived:
            if ((jj & 31) == 32 - kL2Ahead) {
              int32_t yt[8];
              to_rows_quiet(rs, t0 + jj + kL2Ahead, pgn, yt);
              yn = yt[0];
            }
            // tile jj + kL2Ahead into L2, so that its ring load finds it there
            const int32_t ja = jj + kL2Ahead;
            const int32_t ya = __shfl_sync(0xffffffffu, (ja & 31) > (jj & 31) ? yc[0] : yn, ja & 31);
            if (lane == 0 && ja < nt && ya >= 0) {
              tma_prefetch_3d(&tmap_kv4, 0, ya, kOwnChunks * (int)rank);
              tma_prefetch_2d(&tmap_kv64, 2 * kOwnChunks * kChunkDims + kRopeHalf * (int)rank, ya);
            }
            // past this segment's end: the next segment's first tiles
            if (ja >= nt && has_next && ja - nt < nt2 && ja - nt < 32) {
              if (!next_rows) {
                int32_t yt[8];
                to_rows_quiet(u2 % a.n_held, t02, pgf, yt);
                y_next = yt[0];
                next_rows = true;
              }
              const int32_t yb = __shfl_sync(0xffffffffu, y_next, ja - nt);
              if (lane == 0 && yb >= 0) {
                tma_prefetch_3d(&tmap_kv4, 0, yb, kOwnChunks * (int)rank);
                tma_prefetch_2d(&tmap_kv64, 2 * kOwnChunks * kChunkDims + kRopeHalf * (int)rank, yb);
              }
            }
          }
          Boxes cur;
          if (nbox == 1) {
            cur.y[0] = __shfl_sync(0xffffffffu, yc[0], jj & 31);
            cur.bytes = cur.y[0] >= 0 ? kTile * 128 : 0;
          } else {
            int32_t y[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) y[q] = __shfl_sync(0xffffffffu, yc[q], jj & 31);
            make_boxes(y, cur);
          }
          ok = load_tile(cur);
          if (jj == 0) {
            has_next = nx.next(&u2, &t02, &nt2, &wh2, &ks2);
            if (has_next) {
              bool bad2 = false;
              nvis_f = unit_nvis_max(a, u2 / a.n_held, u2 % a.n_held, &bad2);
              fetch_batch(u2 / a.n_held, INT64_MAX, t02, t02 + nt2, pgf);
            }
          }
        }
        it = nx;  // the segment just peeked (its fields below)
        have = has_next;
        u = u2, t0 = t02, nt = nt2, whole = wh2, kslot = ks2;
      }
      // Drain: every slot's last release (a tensor-core commit) lands before the
      // CTA may retire.  Bounded; skipped after an abort.
      if (ok) {
        for (uint32_t s = 0; s < (uint32_t)nts && s < ntiles_cta; ++s) {
          const uint32_t last = s + ((ntiles_cta - 1 - s) / nts) * nts;  // last tile in slot s
          if (!warp_wait(&tempty[s], (last / nts) & 1, abort_s, lane)) break;
        }
      }
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------------ QK issuer
    if (lane == 0 && lo < hi) {
      const uint32_t idesc_qk = idesc_bf16_f32(128, kTile, 0, 0);
      const uint64_t kdesc0 = sw128_desc(smem_u32(ring), 16, 1024);
      const uint64_t qcdesc0 = sw128_desc(smem_u32(qc_s), 16, 1024);
      const uint64_t qrdesc0 = sw64_desc(smem_u32(qr_s), 512);
      const uint64_t rdesc0 = sw64_desc(smem_u32(ring + kRopeOff), 512);
      // QK(j): query chunks 4r, 4r + 1 from TMEM (8 MMAs), chunks 4r + 2, 4r + 3
      // and the rope half from shared memory (8 + 2 MMAs), back to back.
      auto issue_qk = [&](uint32_t j, uint32_t ts) {
        const uint32_t d = tmem + kSCol + kTile * (j & 1);
        const uint32_t soff = (ts * kSlotBytes) >> 4;
        const uint64_t kd = kdesc0 + soff;
#pragma unroll
        for (int i = 0; i < kQTmemChunks; ++i)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_bf16_ts(d, tmem + kQCol + 32 * i + 8 * kk, kd + i * (kChunkBytes >> 4) + 2 * kk, idesc_qk,
                        (i | kk) != 0);
#pragma unroll
        for (int i = kQTmemChunks; i < kOwnChunks; ++i)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_bf16_ss(d, qcdesc0 + (i - kQTmemChunks) * ((128 * 128) >> 4) + 2 * kk,
                        kd + i * (kChunkBytes >> 4) + 2 * kk, idesc_qk, 1);
#pragma unroll
        for (int kk = 0; kk < kRopeHalf / 16; ++kk) mma_bf16_ss(d, qrdesc0 + 2 * kk, rdesc0 + soff + 2 * kk, idesc_qk, 1);
        mma_commit(&bars[kSFull0 + (j & 1)]);
      };
      // Two issuing threads, each blocking in order on its own conditions (no
      // polling loop): lane 0 of this warp issues QK(j) once tile j has landed
      // and the S tile it writes (last used by tile j - 2) has been read; lane 0
      // of warp kPvWarp issues PV(j) once P(j) is ready.  Both feed the same
      // in-order tensor pipe; each commit tracks its own thread's products.
      uint32_t ts_q = 0, ph_q = 0;  // ring slot of the next QK product and its use parity
      SegIter itq;
      itq.init(a.tile_start, U, lo, hi);
      int32_t uq, t0q, ntq, ksq;
      bool wq;
      uint32_t jq = 0;
      int q_seg = 0;
      bool ok = true;
      while (ok && itq.next(&uq, &t0q, &ntq, &wq, &ksq)) {
        for (int q_jj = 0; q_jj < ntq; ++q_jj, ++jq) {
          if (!mbar_wait(&bars[kSFree0 + (jq & 1)], ((jq >> 1) & 1) ^ 1, abort_s) ||
              (q_jj == 0 && !mbar_wait(&bars[kQFull], q_seg & 1, abort_s)) || !mbar_wait(&tfull[ts_q], ph_q, abort_s)) {
            ok = false;
            break;
          }
          tc_fence_after();
          issue_qk(jq, ts_q);
          if (++ts_q == (uint32_t)nts) {
            ts_q = 0;
            ph_q ^= 1;
          }
          if (q_jj == ntq - 1) mma_commit(&bars[kQEmpty]);
        }
        ++q_seg;
      }
    }
  } else if (warp == kPvWarp) {
    // ------------------------------------------------------------------ PV issuer
    if (lane == 0 && lo < hi) {
      const uint32_t idesc_pv = idesc_bf16_f32(128, 256, 0, 1);
      const uint64_t vdesc0 = sw128_desc(smem_u32(ring), kChunkBytes, 1024);
      SegIter itp;
      itp.init(a.tile_start, U, lo, hi);
      int32_t up, t0p, ntp, ksp;
      bool wp;
      uint32_t jp = 0, ts_p = 0;
      int p_seg = 0;
      bool ok = true;
      while (ok && itp.next(&up, &t0p, &ntp, &wp, &ksp)) {
        for (int p_jj = 0; p_jj < ntp; ++p_jj, ++jp) {
          // P(j) ready; the first product of a segment also needs the previous
          // segment's O read out
          if (!mbar_wait(&bars[kPFull0 + (jp & 1)], (jp >> 1) & 1, abort_s) ||
              (p_jj == 0 && p_seg >= 1 && !mbar_wait(&bars[kOFree], (p_seg - 1) & 1, abort_s))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t pa = tmem + kPCol + 32 * (jp & 1);  // P(j): 64 bf16 = 32 columns
          const uint64_t vd = vdesc0 + ((ts_p * kSlotBytes) >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_bf16_ts(tmem + kOCol, pa + 8 * kk, vd + kk * (2048 >> 4), idesc_pv, !(p_jj == 0 && kk == 0));
          mma_commit(&tempty[ts_p]);
          mma_commit(&bars[kPVDone0 + (jp & 1)]);
          if (++ts_p == (uint32_t)nts) ts_p = 0;
        }
        ++p_seg;
      }
    }
  } else if (warp < 8 && 32 * (warp & 3) + kHalfRows * (warp >> 2) < Rg) {
    // ------------------------------------------------------------------ score exchange, softmax, epilogue
    // Warp w < 8 serves the 16 rows [r0, r0 + 16), r0 = 32 (w % 4) + 16 (w / 4),
    // with two threads per row: thread t takes row r0 + t % 16 and keys
    // [32 (t / 16), 32 (t / 16) + 32) of each tile (O columns [128 (t / 16), +128)).
    // Per tile j it reads its rows of this CTA's partial scores S_j^r, adds the
    // peer's (landed in buffer (j & 1) ^ 1) and runs the online softmax.  It also
    // ships its rows of S_j^r to the peer, from the registers it has just read
    // them into: staged in buffer j & 1 and sent with one bulk copy.  The buffer
    // is free: this warp read the peer's tile j - 1 out of it in the previous
    // tile, and my copy of tile j - 1 out of the peer's buffer had landed by
    // then.  Both conditions are local, so no barrier guards the buffers.
    // (Shipping S_{j+1} early, right after that read, was measured slower: the
    // extra TMEM read and staging sit in the middle of the softmax.)
    // Waits are warp-wide and bounded, so a timeout drains every thread.
    const int r0 = 32 * (warp & 3) + kHalfRows * (warp >> 2);
    const int ch = warp;  // exchange channel
    const int h = lane >> 4;
    const int row = r0 + (lane & 15);
    const uint32_t lane_addr = (uint32_t)r0 << 16;
    const uint32_t xrow = (uint32_t)row * kXRowBytes;
    if (lo < hi) {
      auto wwait = [&](uint64_t* bar, uint32_t parity) -> bool { return warp_wait(bar, parity, abort_s, lane); };
      auto wwait_cluster = [&](uint64_t* bar, uint32_t parity) -> bool {
        return warp_wait_cluster(bar, parity, abort_s, lane);
      };
      const uint32_t peer = rank ^ 1u;
      const uint32_t x_peer = mapa_shared(smem_u32(x_s), peer);
      const uint32_t xfull_peer = mapa_shared(smem_u32(&bars[kXFull + ch]), peer);
      // this warp's rows of S_js (in registers) -> buffer js & 1 -> the peer's buffer (js & 1) ^ 1
      auto send = [&](uint32_t js, const uint32_t (&sv)[32]) {
        const uint32_t sb = js & 1;
        const uint32_t dst = smem_u32(x_s) + sb * sl.xbuf + xrow;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          st_shared_v4(dst + ((uint32_t)((8 * h + i) ^ (row & 15)) << 4), sv[4 * i], sv[4 * i + 1], sv[4 * i + 2],
                       sv[4 * i + 3]);
        fence_proxy_async_smem();  // the copy engine reads the staged rows
        __syncwarp();
        if (lane == 0)
          bulk_copy_to_peer(x_peer + (sb ^ 1) * sl.xbuf + (uint32_t)r0 * kXRowBytes,
                            x_s + sb * sl.xbuf + (uint32_t)r0 * kXRowBytes, kHalfRows * kXRowBytes,
                            xfull_peer + 8 * 8 * (sb ^ 1));
      };
      SegIter it;
      it.init(a.tile_start, U, lo, hi);
      int32_t u, t0, nt, kslot;
      bool whole;
      uint32_t jglob = 0;
      int seg = 0;
      bool ok = true;
      const int grow = g * Rg + row;
      const bool has_row = row < Rg && grow < a.R_total;
      // this warp's rows of the query chunks 4r, 4r + 1 (thread t: chunk t / 16 of
      // its row) for request b
      auto q_src = [&](int bq) {
        return reinterpret_cast<const uint4*>(a.q + ((int64_t)bq * a.R_total + grow) * kDk + 256 * (int)rank +
                                              kChunkDims * h);
      };
      // ... into TMEM for segment sq, once QK of segment sq - 1 no longer reads them
      auto load_q = [&](int bq, int sq) -> bool {
        if (!wwait(&bars[kQEmpty], (sq & 1) ^ 1)) return false;
        tc_fence_after();
        const uint4* src = q_src(bq);
        uint32_t r[32];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          uint4 w4 = has_row ? __ldg(src + k) : make_uint4(0, 0, 0, 0);
          r[4 * k] = w4.x; r[4 * k + 1] = w4.y; r[4 * k + 2] = w4.z; r[4 * k + 3] = w4.w;
        }
        tmem_st16x2<32>(tmem + lane_addr + kQCol, r);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kQFull]);
        return true;
      };
      bool q_next = false;  // the next segment's query is already in TMEM
      // Each segment's description and length come from the segment before it
      // (peeked and loaded there), so a segment start waits on no global load.
      bool have = it.next(&u, &t0, &nt, &whole, &kslot);
      int64_t S_cur = have ? a.seq_lens[u / a.n_held] : 0;
      while (ok && have) {
        const int b = u / a.n_held, rs = u % a.n_held;
        if (!q_next && !load_q(b, seg)) { ok = false; break; }
        q_next = false;
        ++seg;
        // The next segment, peeked once this segment's first tile is done (the
        // peek waits on the unit table): its length is loaded then, its query
        // rows go into L2 then and into TMEM before this segment's epilogue, so
        // that its first QK product overlaps the epilogue.
        SegIter nx = it;
        int32_t u2 = 0, t02 = 0, nt2 = 0, ks2 = 0;
        bool wh2 = false, has_next = false;
        int64_t S_next = 0;
        const int64_t S = S_cur;
        int64_t nvis = 0;  // keys of this shard visible to the row
        if (has_row && S >= a.q_len) nvis = count_of(a.shard_begin + rs, S - a.q_len + grow / a.H + 1, a.L);
        float m_ref = -INFINITY;  // running maximum of the row (log2 units)
        float l = 0.f;            // this thread's half of the row's running sum
        float l_row = 0.f;        // the row's running sum
        for (int jj = 0; jj < nt; ++jj, ++jglob) {
          const uint32_t j = jglob, bsel = j & 1, rb = bsel ^ 1;
          // ---- this CTA's partial scores of tile j
          uint32_t s[32];  // score bits, keys [32 h, 32 h + 32)
          if (!wwait(&bars[kSFull0 + bsel], (j >> 1) & 1)) { ok = false; break; }
          tc_fence_after();
          tmem_ld16x2_sync<32>(tmem + lane_addr + kSCol + kTile * bsel, s);
          send(j, s);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[kSFree0 + bsel]);
          // ---- the peer's partial scores of tile j: S = mine + peer's
          if (!wwait_cluster(&bars[kXFull + 8 * rb + ch], (j >> 1) & 1)) { ok = false; break; }
          {
            const uint32_t src = smem_u32(x_s) + rb * sl.xbuf + xrow;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint4 w4 = ld_shared_v4(src + ((uint32_t)((8 * h + i) ^ (row & 15)) << 4));
              const uint64_t a0 = f2_add(f2_pack(s[4 * i], s[4 * i + 1]), f2_pack(w4.x, w4.y));
              const uint64_t a1 = f2_add(f2_pack(s[4 * i + 2], s[4 * i + 3]), f2_pack(w4.z, w4.w));
              f2_unpack(a0, s[4 * i], s[4 * i + 1]);
              f2_unpack(a1, s[4 * i + 2], s[4 * i + 3]);
            }
          }
          __syncwarp();  // every lane's reads of buffer rb are done
          if (lane == 0 && j + 2 < ntiles_cta)
            mbar_arrive_expect_tx(&bars[kXFull + 8 * rb + ch], kHalfRows * kXRowBytes);
          // ---- online softmax of tile j
          const int64_t lim = nvis - ((int64_t)(t0 + jj) * kTile + 32 * h);  // keys k < lim are visible
          if (lim < 32) {
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (k >= lim) s[k] = __float_as_uint(-INFINITY);
          }
          float mx[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) mx[k] = __uint_as_float(s[k]);
#pragma unroll
          for (int k = 4; k < 32; k += 2)
            mx[((k - 4) >> 1) & 3] = fmax3(mx[((k - 4) >> 1) & 3], __uint_as_float(s[k]), __uint_as_float(s[k + 1]));
          float mraw = fmax3(mx[0], mx[1], fmaxf(mx[2], mx[3]));
          mraw = fmaxf(mraw, __shfl_xor_sync(0xffffffffu, mraw, 16));  // the row's other 32 keys
          const float mt = mraw * a.scale_log2;  // scale > 0: the max commutes with the scaling
          bool need = false;
          float alpha = 1.f;
          if (m_ref == -INFINITY) {
            m_ref = mt;  // nothing accumulated yet for this row
          } else if (mt > m_ref + kRescaleThreshold) {
            need = true;
            alpha = exp2f(m_ref - mt);
            m_ref = mt;
          }
          if (__any_sync(0xffffffffu, need)) {
            // rows whose maximum moved: scale their O row once PV(j - 1) is done
            // (a row's maximum is finite only after a tile of this segment, so j >= 1)
            if (!wwait(&bars[kPVDone0 + ((j - 1) & 1)], ((j - 1) >> 1) & 1)) { ok = false; break; }
            tc_fence_after();
            rescale_rows(tmem + lane_addr + kOCol, alpha);
          }
          const float m_use = (m_ref == -INFINITY) ? 0.f : m_ref;
          const float cs = a.scale_log2;
          const uint64_t cs2 = f2_pack(__float_as_uint(cs), __float_as_uint(cs));
          const uint64_t nm2 = f2_pack(__float_as_uint(-m_use), __float_as_uint(-m_use));
          uint64_t ps[4] = {0, 0, 0, 0};  // pairs of partial row sums (+0.f bits)
          uint32_t pk[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            uint32_t x0, x1;
            f2_unpack(f2_fma(f2_pack(s[2 * k], s[2 * k + 1]), cs2, nm2), x0, x1);
            const float p0 = fast_exp2(__uint_as_float(x0));
            const float p1 = fast_exp2(__uint_as_float(x1));
            ps[k & 3] = f2_add(ps[k & 3], f2_pack(__float_as_uint(p0), __float_as_uint(p1)));
            __nv_bfloat162 hh = __floats2bfloat162_rn(p0, p1);
            pk[k] = *reinterpret_cast<uint32_t*>(&hh);
          }
          {
            uint32_t a0, a1;
            f2_unpack(f2_add(f2_add(ps[0], ps[1]), f2_add(ps[2], ps[3])), a0, a1);
            l = l * alpha + (__uint_as_float(a0) + __uint_as_float(a1));
          }
          // P(j) -> TMEM (A operand of the PV product) once PV(j - 2) has read the buffer
          if (j >= 2 && !wwait(&bars[kPVDone0 + bsel], ((j - 2) >> 1) & 1)) { ok = false; break; }
          tc_fence_after();
          tmem_st16x2_16<16>(tmem + lane_addr + kPCol + 32 * bsel, pk);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[kPFull0 + bsel]);
          if (jj == 0) {
            has_next = nx.next(&u2, &t02, &nt2, &wh2, &ks2);
            if (has_next) {
              S_next = a.seq_lens[u2 / a.n_held];
              if (has_row) asm volatile("prefetch.global.L2 [%0];" ::"l"(q_src(u2 / a.n_held)));
            }
          }
        }
        if (!ok) break;
        if (has_next) {
          if (!load_q(u2 / a.n_held, seg)) { ok = false; break; }
          q_next = true;
        }
        l_row = l + __shfl_xor_sync(0xffffffffu, l, 16);
        // ---------------- epilogue: O rows / l -> o (this CTA's 256 dims), lse
        const uint32_t jl = jglob - 1;
        if (!wwait(&bars[kPVDone0 + (jl & 1)], (jl >> 1) & 1)) { ok = false; break; }
        tc_fence_after();
        const int rows_here = min(Rg, a.R_total - g * Rg);
        const bool writes = row < rows_here;
        const int64_t out_base = ((int64_t)rs * a.B + b) * a.R_total + g * Rg;
        const int64_t piece_base = (int64_t)(2 * v + kslot) * a.R_total + g * Rg;
        const int64_t out_row = out_base + row, piece_row = piece_base + row;
        const float inv = l_row != 0.f ? 1.f / l_row : 0.f;  // 0: no key seen; a NaN stays one
        // staging for the fp32 rows: this warp's rows of the buffer the last tile's
        // peer scores were read from
        store_o_rows(a, tmem + lane_addr + kOCol, rows_here, whole, out_base, piece_base, r0, 256 * (int)rank + 128 * h,
                     inv, smem_u32(x_s) + ((jl & 1) ^ 1) * sl.xbuf + (uint32_t)r0 * kXRowBytes);
        if (writes && h == 0 && rank == 0) {
          const float lse2 = l_row != 0.f ? m_ref + log2f(l_row) : -INFINITY;
          if (whole)
            a.lse_part[out_row] = a.base2 ? lse2 : lse2 * kLn2;
          else
            a.piece_lse[piece_row] = lse2;
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
  }
  else if (warp < 8) {
    // No rows of the group: zero this warp's 16 TMEM lanes of the P and query
    // columns once, so the M = 128 products carry zeros, not stale data, in the
    // padding rows (their results are never read).
    const uint32_t zl = (uint32_t)(32 * (warp & 3) + kHalfRows * (warp >> 2)) << 16;
    uint32_t z[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) z[i] = 0u;
    tmem_st16x2<32>(tmem + zl + kPCol, z);
    tmem_st16x2<32>(tmem + zl + kQCol, z);
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

// ---------------------------------------------------------------------------- host side
PairKernel g_kernel(reinterpret_cast<const void*>(&partial_tc_kernel), kThreads);

bool make_plan(const dcp_layout_t* layout, int n_held, int B, int q_len, int H, Plan* p) {
  plan_groups(q_len, H, p);
  int nts = (int)((kSmemBudget - smem_layout(p->Rg, 0).total) / kSlotBytes);
  if (nts > kMaxTileSlots) nts = kMaxTileSlots;
  p->nts = nts;
  p->smem = smem_layout(p->Rg, nts).total;
  return nts >= 3 && plan_ranges(layout, n_held, B, q_len, H, g_kernel, p);
}

// bf16 [rows, 576] seen as [9 chunks][rows][64 dims] (dims innermost, then rows,
// then chunks 128 bytes apart): boxes of [4 chunks][box_rows][64] land as four
// consecutive 128-byte-swizzled [box_rows][64] tiles.
bool make_tmap_chunks(CUtensorMap* m, const void* base, uint64_t rows, uint32_t box_rows) {
  auto enc = tmap_encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)kChunkDims, (cuuint64_t)rows, (cuuint64_t)(kDk / kChunkDims)};
  cuuint64_t strides[2] = {(cuuint64_t)kDk * 2, (cuuint64_t)kChunkDims * 2};
  cuuint32_t box[3] = {(cuuint32_t)kChunkDims, box_rows, (cuuint32_t)kOwnChunks};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tensor maps and launches of one partial decode on a checked plan and workspace.
int32_t launch_bf16(const Plan& p, const DecodeCall& c, void* workspace) {
  const TcArgs a = device_args(p, c, workspace);
  const uint64_t q_rows = (uint64_t)c.B * a.R_total, kv_rows = (uint64_t)a.n_held * a.pool_rows;
  CUtensorMap tq, tkv, tq64, tkv64, tkv4;
  if (!make_tmap(&tq, c.q, q_rows, (uint32_t)p.Rg)) return DCP_ERR_CUDA;
  if (!make_tmap(&tkv, c.arena, kv_rows, (uint32_t)p.box_rows)) return DCP_ERR_CUDA;
  if (!make_tmap(&tq64, c.q, q_rows, (uint32_t)p.Rg, true)) return DCP_ERR_CUDA;
  if (!make_tmap(&tkv64, c.arena, kv_rows, (uint32_t)p.box_rows, true)) return DCP_ERR_CUDA;
  if (!make_tmap_chunks(&tkv4, c.arena, kv_rows, (uint32_t)p.box_rows)) return DCP_ERR_CUDA;
  if (!g_kernel.ensure_smem(p.smem)) return DCP_ERR_CUDA;
  return launch_decode(p, a, kThreads, c.stream, [&](const cudaLaunchConfig_t& lc) {
    return cudaLaunchKernelEx(&lc, partial_tc_kernel, tq, tkv, tq64, tkv64, tkv4, a);
  });
}

}  // namespace

extern "C" size_t dcp_mla_decode_workspace_size(const dcp_layout_t* layout, int32_t shard_begin,
                                                int32_t shard_end, int32_t B, int32_t q_len, int32_t H) {
  Plan p;
  if (!size_args_ok(layout, shard_begin, shard_end, B, q_len, H) ||
      !make_plan(layout, shard_end - shard_begin, B, q_len, H, &p))
    return 0;
  return p.ws_total;
}

extern "C" int32_t dcp_mla_decode_partial(const dcp_layout_t* layout, int32_t shard_begin, int32_t shard_end,
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
  return rc != DCP_OK ? rc : launch_bf16(p, c, workspace);
}

// ---------------------------------------------------------------------------- allocation-free variant
// Some callers cannot hand the library a workspace: a serving process that has
// given every free byte of HBM to its KV pool and forbids further device
// allocations, or a plain C host with no device-memory manager of its own.
// For them the partial decode can run on a scratch area that the library owns:
// a file-scope device array, created when the library is loaded on a device and
// kept until the process exits.
namespace {

constexpr size_t kStaticScratchBytes = size_t(64) << 20;  // 64 MiB per device
__device__ __align__(256) unsigned char g_partial_scratch[kStaticScratchBytes];

std::mutex g_scratch_mutex;
void* g_scratch_addr[kMaxDevices] = {};

// Device address of g_partial_scratch on the current device (looked up once per
// device; in host code the array's name is only a host-side stand-in).
void* scratch_address() {
  const int dev = current_device();
  if (dev < 0) return nullptr;
  std::lock_guard<std::mutex> lock(g_scratch_mutex);
  if (!g_scratch_addr[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_partial_scratch) != cudaSuccess) return nullptr;
    g_scratch_addr[dev] = p;
  }
  return g_scratch_addr[dev];
}

}  // namespace

extern "C" size_t dcp_mla_decode_static_scratch_bytes(void) { return kStaticScratchBytes; }

extern "C" int32_t dcp_mla_decode_partial_static(const dcp_layout_t* layout, int32_t shard_begin, int32_t shard_end,
                                                 const void* q, int32_t B, int32_t q_len, int32_t H,
                                                 const void* arena, int64_t pool_pages,
                                                 const int32_t* block_table, int64_t bt_stride, int64_t max_pages,
                                                 const int64_t* seq_lens, float scale, int32_t lse_base,
                                                 void* o_part, int32_t o_part_dtype, float* lse_part,
                                                 int32_t* status, void* stream) {
  const DecodeCall c{layout, shard_begin, shard_end, q, B, q_len, H, arena, pool_pages, block_table, bt_stride,
                     max_pages, seq_lens, scale, lse_base, o_part, o_part_dtype, lse_part, status, stream};
  const int32_t rc = check_decode_args(c);
  if (rc != DCP_OK) return rc;
  Plan p;
  if (!make_plan(layout, shard_end - shard_begin, B, q_len, H, &p)) return DCP_ERR_CUDA;
  if (p.ws_total > kStaticScratchBytes) return DCP_ERR_TOO_LARGE;
  void* ws = scratch_address();
  return ws ? launch_bf16(p, c, ws) : DCP_ERR_CUDA;
}
