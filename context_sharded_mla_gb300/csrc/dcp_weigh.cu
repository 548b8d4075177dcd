// dcp_weigh.cu — the attention weight of every cached row, summed over a call's queries:
//
//   w[r][b][i] = decay * w[r][b][i] + sum_{rows (t, h) that see p} exp2(c * q . k_i - lse2[t, h])
//
// Sources: "MLA 的 Decode Context Parallelism", section 2 (576-d single-head scores);
// lse is the merged one, so no maximum and no second pass are needed.
//
// The product is laid out with the KEYS on the accumulator's lanes and the query rows on
// its columns: a key's whole sum is then one thread's, over its own TMEM lane, in a fixed
// order, and a key that must not count (past the length, NaN) touches no other.
//
// A pair of CTAs (two SMs) holds up to 256 query rows in shared memory, half in each, and
// runs one product of 256 keys x Rg rows (cta_group::2): each SM brings 128 keys of its
// own and reads the other half of the queries from its peer.  Per SM and tile that is
// 147 KB of keys for 128 * Rg * 576 multiply-adds: memory-bound up to about 256 rows (2 *
// 576 * Rg flop for 1152 bytes against 280 flop/byte), tensor-bound above.  Keys stream
// through a ring of 16-KB chunks (128 keys x 64 dims); the chunks of a tile are consumed
// in order, so a product starts when its first chunk is there.
//
// More than 256 rows: groups of at most 256, one after the other.  The nine chunks of a
// tile's keys then stay, each replaced when the last group is done with it, and the queries
// (which the L2 holds) pass through the ring: 4 requests of 128k tokens with 64 queries of
// 96 heads take 1950-1985 us.  With the queries held over blocks of tiles that later groups
// find in the L2 2067 at best (two pair-tiles; 2309 with four, 2132 with one).
//
// The 4-bit cache: 416-byte rows land raw, eight warps turn them (a lane a key, 128 dims at
// a time) into bf16 operands and write them to TMEM, where the product takes its A operand
// from (lanes are keys there too); no dequantised tile is stored.  Groups of 128 rows; the
// queries are held, over blocks of eight pair-tiles (65 MB over the card, for the L2): 32
// requests of 32k tokens with 8 queries of 128 heads take 871 us, with four 931, sixteen 891.
//
// Work: the pair-tiles (2 x 128 rows of one request) of all requests in a row, cut into as
// many equal runs as there are pairs.  A run's start is found from the lengths by every
// CTA for itself (a block-wide scan), so the call is one launch with no workspace.
// Many query rows over few tiles are cut between row groups as well: the pair that begins
// a tile writes its weights, the others leave their sums in a workspace and a second
// launch adds them, in order.  64 queries of 96 heads over 2 x 32k tokens 249 -> 218 us,
// 61 of 128 over 8k 81 -> 47, 4-bit 32 of 128 over 4k 99 -> 34.
#include "dcp_decode.cuh"

namespace {

constexpr int kKeys = 128;                 // keys a CTA brings to a tile
constexpr int kChunks = kDk / kChunkDims;  // 9
constexpr int kStageBytes = kKeys * 128;   // 16 KB: 128 keys x 64 dims
constexpr int kMaxStages = 12;
constexpr int kBlockQ4 = 8;                // 4-bit: pair-tiles of a block when there is more than one row group
constexpr int kRawTile = kKeys * kQ4RowBytes;
constexpr int kMaxRaw = 3;
// The tensor core cuts its running sum off toward zero at each of the 36 steps of a score instead of rounding it.  Of a
// bf16 score that loses, in 2^-24 of it: 9 to 10 where queries and rows are dense, 20 where all products have one sign, under
// 1 with few terms (measured against fp64).  8 are made good: a dense query row's weights then sum to one within 2 against fp64
// and within 5 under the decode's own lse (the decode adds two sums of 18 steps and loses half as much); without that 10 and
// 5, with the difference to the decode alone (5) 5 and 1.  At worst, one sign or few terms: 12 and 8; without 20 and 11.
// 4-bit values have few bits, of which the sums cut fewer: dense 4, within 2 of the decode's.  Left as it is (made good
// like the bf16 ones they summed to 4 to 5 too much against fp64 and 7 under the decode's lse).
constexpr double kTruncation = 0x1p-21;
// 4-bit: operand slots of 128 dims (64 columns) in TMEM.  A slot of 64 dims costs its wait, its commit and its
// products' issue more than the products take at 128 rows.
constexpr int kASlots = 4;
constexpr int kAParts = 5;                 // slots a tile fills: 4 of codes, one of the 64 position dims
constexpr int kACol = 256;
constexpr uint32_t kAllCols = 512;

// Warps: 0-3 sums, 4 keys in, 5 products, 6 queries in, 7 idle or keys in too; 4-bit: 8-15 dequantise, two sets of four that take
// slots in turn.  With three 128 us against 117 (32 requests of 32k tokens, 128 heads), with four 135;
// both sets on every slot, 64 dims each: 128 (a warp's waits for its slots are then twice as many).
constexpr int kDequantSets = 2;
constexpr int kKeyWarp = 4, kMmaWarp = 5, kQueryWarp = 6, kKeyWarp2 = 7, kDequantWarp = 8;
constexpr int kThreads = 256, kThreadsQ4 = kThreads + 128 * kDequantSets;

struct WeighArgs {
  Layout L;
  int32_t shard_begin, n_held;
  int32_t B, q_len, H, R;       // R = q_len * H
  int32_t Rg, ngroups;          // columns a group, groups
  int32_t stages;               // ring stages, or raw tiles (4-bit)
  int32_t held_bytes, ring_bytes;  // of a held chunk, of a stage
  int32_t box_rows, nbox;       // rows a copy (min(P, 64)), copies a tile
  int32_t npairs;
  int32_t block;                // most pair-tiles of a block
  // what pairs add to a tile that another pair has begun (null: no tile is shared)
  int64_t* units;               // units of the call
  int64_t* part_at;             // [pairs, 256] entry of weights, -1: none
  float* part;                  // [pairs, 256]
  int64_t pool_rows, pool_pages, max_rows;
  const unsigned char* arena;
  const int32_t* bt;
  int64_t bt_stride, max_pages;
  const int64_t* seq_lens;
  float scale_log2;
  int32_t base2;
  const float* lse;
  const int64_t* old_lens;
  float decay;
  float* weights;
  int64_t w_stride;
  int32_t* status;
};

// ---------------------------------------------------------------- pair forms of the PTX wrappers
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar_cluster, int32_t x,
                                                 int32_t y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
      "%4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void expect_tx_cluster(uint32_t bar_cluster, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;" ::"r"(bar_cluster),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void arrive_cluster(uint32_t bar_cluster) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}
__device__ __forceinline__ void mma_pair_ss(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_pair_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(
          d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(acc)
      : "memory");
}
// Arrive on the barrier at this offset in both CTAs once this thread's products so far are complete.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

// warp_wait for waits that are long as a rule: the warp sleeps in the barrier, up to kSuspendNs at a time, instead of
// asking again and again (the other warps want the issue slots).  Bounded as mbar_wait is.
__device__ __forceinline__ bool sleep_wait(uint64_t* bar, uint32_t parity, volatile int* abort_s) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const uint64_t t0 = globaltimer();
  while (true) {
    if (__all_sync(0xffffffffu, mbar_try_wait_for(bar, parity, kSuspendNs))) return true;
    if (__any_sync(0xffffffffu, *abort_s)) return false;
    if (__any_sync(0xffffffffu, globaltimer() - t0 > kWaitLimitNs)) {
      *abort_s = 1;
      return false;
    }
  }
}

// ---------------------------------------------------------------- barriers and shared memory
enum : int {
  kFull = 0,                            // stage of the ring full in both CTAs (bf16; counted at the leader)
  kEmpty = kFull + kMaxStages,          // its products are done
  kHeldFull = kEmpty + kMaxStages,      // held chunk there in both CTAs (at the leader)
  kHeldEmpty = kHeldFull + kChunks,
  kSFull = kHeldEmpty + kChunks,        // scores of a tile
  kSFree = kSFull + 2,                  // read by the sums' warps of both CTAs (at the leader)
  kAFull = kSFree + 2,                  // 4-bit: operand slot written in both CTAs (at the leader)
  kAEmpty = kAFull + kASlots,
  kRFull = kAEmpty + kASlots,           // 4-bit: raw tile landed
  kRFree = kRFull + kMaxRaw,
  kNumBars = kRFree + kMaxRaw
};

struct Smem {
  uint32_t held, ring, bars, lse, acc, misc, total;
};
// The held chunks, the ring, barriers, lse of the rows of two groups, a block's sums (4-bit), the rest.
__host__ __device__ inline Smem smem_of(int held_bytes, int stages, int ring_bytes, bool q4) {
  Smem s;
  s.held = 0;
  s.ring = (uint32_t)kChunks * held_bytes;
  s.bars = s.ring + (uint32_t)stages * ring_bytes;
  s.lse = s.bars + (kNumBars * 8 + 15) / 16 * 16;
  s.acc = s.lse + 2 * 256 * 4;
  s.misc = s.acc + (q4 ? kBlockQ4 * kKeys * 4 : 0);
  s.total = s.misc + 128;
  return s;
}

// The slots that a role fills one after the other, held or of the ring.
struct Slots {
  uint64_t* empty;
  uint32_t full;     // the leader's barriers, by cluster address
  uint32_t at0, bytes, n;
  uint32_t at = 0, ph = 0, uses = 0;
  __device__ bool wait(volatile int* abort_s) const { return sleep_wait(empty + at, ph ^ 1, abort_s); }
  __device__ uint32_t full_bar() const { return full + 8 * at; }
  __device__ uint32_t dst() const { return at0 + at * bytes; }
  __device__ void advance() {
    ++uses;
    if (++at == n) {
      at = 0;
      ph ^= 1;
    }
  }
  // every slot's last release lands before the CTA may leave
  __device__ void drain(volatile int* abort_s) const {
    for (uint32_t s = 0; s < n && s < uses; ++s)
      if (!sleep_wait(empty + s, ((uses - 1 - s) / n) & 1, abort_s)) return;
  }
};

// ---------------------------------------------------------------- work
// Rows of a request on the shards, from one division.
struct Shape {
  int64_t S, full, rem;  // S = full / I * (N * I) + rem
  __device__ void set(const WeighArgs& a, int64_t S_) {
    S = S_;
    const int64_t blk = a.L.N * a.L.I;
    const int64_t k = S_ > 0 ? div_tiles(S_, blk) : 0;
    full = k * a.L.I;
    rem = S_ > 0 ? S_ - k * blk : 0;
  }
  __device__ int64_t count(const WeighArgs& a, int rs) const {
    int64_t x = rem - (a.shard_begin + rs) * a.L.I;
    x = x < 0 ? 0 : (x > a.L.I ? a.L.I : x);
    return full + x;
  }
  __device__ int32_t rows(const WeighArgs& a, int rs) const {  // none of a request shorter than its queries
    if (S < a.q_len) return 0;
    const int64_t n = count(a, rs);
    return (int32_t)(n < a.max_rows ? n : a.max_rows);
  }
  __device__ int32_t tiles(const WeighArgs& a, int rs) const { return (rows(a, rs) + kKeys - 1) / kKeys; }
  // Shards before `cut` have `full` + I rows, those after it `full`.
  __device__ int32_t pair_tiles(const WeighArgs& a) const {
    if (S < a.q_len) return 0;
    const int32_t cut = (int32_t)max((int64_t)0, min(div_tiles(rem, a.L.I) - a.shard_begin, (int64_t)a.n_held));
    const int32_t most = (int32_t)min(full + a.L.I, a.max_rows), least = (int32_t)min(full, a.max_rows);
    int32_t t = cut * ((most + kKeys - 1) / kKeys);
    if (cut < a.n_held) t += tiles(a, cut) + (a.n_held - cut - 1) * ((least + kKeys - 1) / kKeys);
    return (t + 1) / 2;
  }
};

// Where pair p's units (pair-tile, row group) begin.
__device__ __forceinline__ int64_t run_start(int64_t units, int p, int npairs) { return div_tiles(units * p, npairs); }

// A pair's run, tile by tile: blocks of pair-tiles of one request, and in a block every row
// group in turn.  Each role of a CTA walks it for itself.
struct Walk {
  int32_t b, left;           // request; pair-tiles left, this block's included
  int32_t g0, g1;            // row groups of the block (all but for a tile shared with another pair)
  int32_t g_last;            // groups of the run's last tile
  int32_t pt, npt;           // block's first pair-tile, pair-tiles of the request
  int32_t nblk, g, i;        // pair-tiles of the block, row group, pair-tile within the block
  int32_t rs, t, rows, nt;   // this CTA's tile: shard (n_held: none), tile of it; the shard's rows and tiles
  int32_t rs0, t0, rows0, nt0;  // the same at the block's start
  Shape sh;
  int64_t S_next;            // the next request's length, already loaded

  __device__ void shard(const WeighArgs& a, int32_t r) {
    rs = r;
    rows = r < a.n_held ? sh.rows(a, r) : 0;
    nt = (rows + kKeys - 1) / kKeys;
  }
  __device__ void advance(const WeighArgs& a, int32_t by) {
    t += by;
    while (t >= nt && rs < a.n_held) {
      t -= nt;
      shard(a, rs + 1);
    }
  }
  __device__ void block(const WeighArgs& a, int32_t g_first = 0) {
    nblk = min(left, npt - pt);
    g0 = g_first;
    g1 = a.ngroups;
    if (a.ngroups > 1) {
      nblk = g0 > 0 ? 1 : min(nblk, a.block);
      if (nblk == left && g_last < a.ngroups) {  // the last tile by itself
        if (nblk > 1) --nblk;
        else g1 = g_last;
      }
    }
    g = g0;
    i = 0;
    rs0 = rs;
    t0 = t;
    rows0 = rows;
    nt0 = nt;
  }
  __device__ void request(const WeighArgs& a, int64_t S) {
    sh.set(a, S);
    npt = sh.pair_tiles(a);
    S_next = b + 1 < a.B ? __ldg(a.seq_lens + b + 1) : 0;
  }
  __device__ void start(const WeighArgs& a, int32_t b_, int32_t pt_, int32_t n, int32_t g_first, int32_t g_last_,
                        int rank) {
    left = n;
    g_last = g_last_;
    b = b_;
    pt = pt_;
    request(a, __ldg(a.seq_lens + b));
    t = 0;
    shard(a, 0);
    advance(a, 2 * pt + rank);
    block(a, g_first);
  }
  __device__ bool next(const WeighArgs& a, int rank) {
    if (++i < nblk) {
      advance(a, 2);
      return true;
    }
    i = 0;
    if (++g < g1) {
      rs = rs0;
      t = t0;
      rows = rows0;
      nt = nt0;
      return true;
    }
    left -= nblk;
    pt += nblk;
    if (left <= 0) return false;
    if (pt < npt) {
      advance(a, 2);  // from the last tile of the block
    } else {
      do {
        if (++b >= a.B) return false;
        request(a, S_next);
      } while (npt == 0);
      pt = 0;
      t = 0;
      shard(a, 0);
      advance(a, rank);
    }
    block(a);
    return true;
  }
  __device__ bool group_begins() const { return i == 0; }
  // the held operand is taken up with this tile and group, is done with after them
  template <bool kKeysHeld>
  __device__ bool first() const { return kKeysHeld ? g == g0 : i == 0; }
  template <bool kKeysHeld>
  __device__ bool last() const { return kKeysHeld ? g == g1 - 1 : i == nblk - 1; }
};

// Where copy `box` of the walk's tile starts: its page id, loaded here and looked at later.
__device__ __forceinline__ int32_t box_row(const WeighArgs& a, const Walk& w, int box) {
  if (w.rs >= a.n_held || box >= a.nbox) return -1;
  const int32_t rho = w.t * kKeys + box * a.box_rows;
  return rho < w.rows ? rho : -1;
}
__device__ __forceinline__ int32_t page_of(const WeighArgs& a, const Walk& w, int32_t rho) {
  return rho < 0 ? -1 : __ldg(a.bt + (int64_t)w.b * a.bt_stride + rho / (int32_t)a.L.P);
}
// Its first row over all held pools; -1: nothing to copy (a bad page is flagged).
__device__ __forceinline__ int32_t pool_row(const WeighArgs& a, int32_t rs, int32_t rho, int32_t page) {
  if (rho < 0) return -1;
  if (page < 0 || page >= a.pool_pages) {
    flag(a.status, DCP_STATUS_BAD_PAGE_ID);
    return -1;
  }
  return (int32_t)(rs * a.pool_rows + page * a.L.P + rho % (int32_t)a.L.P);
}

// 32 bytes of shared memory.  (4-bit rows lie 416 bytes apart, so that eight neighbouring lanes meet two to a bank;
// sparing that by a trade of the halves costs more instructions than it is worth.)
__device__ __forceinline__ void load32(uint32_t at, uint32_t* w) {
  const uint4 x = ld_shared_v4(at), y = ld_shared_v4(at + 16);
  w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
  w[4] = y.x; w[5] = y.y; w[6] = y.z; w[7] = y.w;
}
// Four scales (64 dims) and 8 words of codes -> 32 bf16 pairs.
__device__ __forceinline__ void dequant_chunk(const uint32_t (&w)[8], uint32_t four, uint32_t (&v)[32]) {
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t s2[2], off2[2];
    q4_scales(half ? four >> 16 : four & 0xFFFFu, s2, off2);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t p[4];
      q4_values(w[4 * half + k], s2[k >> 1], off2[k >> 1], p);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[16 * half + 4 * k + e] = p[e];
    }
  }
}

// kKeysHeld: the keys of a tile stay and the queries pass through the ring.
template <bool kQ4, bool kKeysHeld>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kQ4 ? kThreadsQ4 : kThreads, 1)
    weigh_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_kv, WeighArgs a) {
  extern __shared__ __align__(1024) unsigned char smem[];
  constexpr int kBlockThreads = kQ4 ? kThreadsQ4 : kThreads, kWarps = kBlockThreads / 32;
  if ((smem_u32(smem) & 1023u) != 0) {  // every CTA of the launch sees the same base: all leave
    if (threadIdx.x == 0) flag(a.status, DCP_STATUS_INTERNAL);
    return;
  }
  const Smem sl = smem_of(a.held_bytes, a.stages, a.ring_bytes, kQ4);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + sl.bars);
  float* lse_s = reinterpret_cast<float*>(smem + sl.lse);
  float* acc_s = reinterpret_cast<float*>(smem + sl.acc);
  uint32_t* tmem_base_s = reinterpret_cast<uint32_t*>(smem + sl.misc);
  volatile int* abort_s = reinterpret_cast<volatile int*>(smem + sl.misc + 4);
  // request, pair-tile, pair-tiles of the run (met in part too), first group of the first, groups of the last, units
  int32_t* start_s = reinterpret_cast<int32_t*>(smem + sl.misc + 8);
  int32_t* warp_sums = reinterpret_cast<int32_t*>(smem + sl.misc + 32);
  static_assert(32 + 4 * kWarps <= 128, "room for them");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster_ctarank();
  const int pair = blockIdx.x >> 1;

  const int32_t per = (a.B + kBlockThreads - 1) / kBlockThreads;  // requests a thread of the scan below
  const int32_t b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
  const int64_t S_first = b0 < b1 ? __ldg(a.seq_lens + b0) : 0;
  static_assert(kNumBars <= kBlockThreads, "a thread a barrier");
  if (tid < kNumBars) {
    const bool two = tid < kEmpty || (tid >= kHeldFull && tid < kHeldEmpty);        // an arrival of each CTA
    const bool eight = tid >= kSFree && tid < kAEmpty;                               // of four warps of each
    mbar_init(&bars[tid], two ? 2 : eight ? 8 : tid >= kRFree ? 4 * kDequantSets : 1);
    fence_barrier_init();
  }
  if (tid == 0) *abort_s = 0;
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_base_s)),
                 "r"(kAllCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  __syncwarp();
  tc_fence_before();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // the barriers are set up
  // ---- this pair's run of pair-tiles: a scan over the requests
  {
    int32_t mine = 0;
    for (int32_t b = b0; b < b1; ++b) {
      Shape sh;
      sh.set(a, b == b0 ? S_first : __ldg(a.seq_lens + b));
      mine += sh.pair_tiles(a);
      if (blockIdx.x == 0) {
        if (sh.S < a.q_len) flag(a.status, DCP_STATUS_BAD_LENGTH);
        else if (sh.full + a.L.I > a.max_rows)  // only then can a shard have more rows than its table
          for (int rs = 0; rs < a.n_held; ++rs)
            if (sh.count(a, rs) > a.max_rows) flag(a.status, DCP_STATUS_BAD_PAGE_ID);
      }
    }
    int32_t incl = mine;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int32_t y = __shfl_up_sync(0xffffffffu, incl, s);
      if (lane >= s) incl += y;
    }
    if (lane == 31) warp_sums[warp] = incl;
    if (tid == 0) start_s[2] = 0;
    __syncthreads();
    int32_t before = incl - mine, total = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += warp_sums[w];
      total += warp_sums[w];
    }
    // the run in units; its tiles and where in the first and last of them it begins and ends
    // Tiles are shared where whole ones would leave a pair 1/16 more than its part.  (4-bit: 5/16 of two tiles and more;
    // the tiles of a shared run are blocks of one, 2.7 us a group where blocks of four take 2.1.)
    const int32_t G = a.ngroups, most = (total + a.npairs - 1) / a.npairs;
    const bool share =
        a.part && 16 * ((int64_t)most * a.npairs - total) > (kQ4 && most > 1 ? 5 : 1) * (int64_t)total;
    const int32_t per_tile = share ? G : 1;
    const int64_t u0 = run_start((int64_t)total * per_tile, pair, a.npairs);
    const int64_t u1 = run_start((int64_t)total * per_tile, pair + 1, a.npairs);
    if (a.part && blockIdx.x == 0 && tid == 0) *a.units = share ? (int64_t)total * G : 0;
    const int32_t lo = (int32_t)(per_tile == 1 ? u0 : div_tiles(u0, G));
    if (u0 < u1 && before <= lo && lo < before + mine) {
      int32_t b = b0, x = lo - before;
      for (; b + 1 < b1; ++b) {  // (with what is left it is the last)
        Shape sh;
        sh.set(a, __ldg(a.seq_lens + b));
        const int32_t n = sh.pair_tiles(a);
        if (x < n) break;
        x -= n;
      }
      const int32_t hi = (int32_t)(per_tile == 1 ? u1 : div_tiles(u1 + G - 1, G));  // tile after the last
      start_s[0] = b;
      start_s[1] = x;
      start_s[2] = hi - lo;
      start_s[3] = per_tile == 1 ? 0 : (int32_t)(u0 - (int64_t)lo * G);
      start_s[4] = per_tile == 1 ? G : (int32_t)(u1 - (int64_t)(hi - 1) * G);
      start_s[5] = per_tile == 1 ? (hi - lo) * G : (int32_t)(u1 - u0);
    }
  }
  __syncthreads();  // the start is known
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  tc_fence_after();
  const uint32_t tmem = *tmem_base_s;
  const uint32_t lead = mapa_shared(smem_u32(bars), 0);  // the leader's barriers
  Walk w;
  const bool any = start_s[2] > 0;
  if (any && (!kQ4 || warp < kDequantWarp)) w.start(a, start_s[0], start_s[1], start_s[2], start_s[3], start_s[4], rank);
  auto slots_of = [&](bool held) -> Slots {
    return held ? Slots{&bars[kHeldEmpty], lead + 8 * kHeldFull, smem_u32(smem) + sl.held, (uint32_t)a.held_bytes, kChunks}
                : Slots{&bars[kEmpty], lead + 8 * kFull, smem_u32(smem) + sl.ring, (uint32_t)a.ring_bytes,
                        (uint32_t)a.stages};
  };

  const bool two = !kQ4 && a.nbox > 4;  // key warps
  if ((warp == kKeyWarp || (two && warp == kKeyWarp2)) && any) {
    // ------------------------------------------------------------------ keys in
    // A lane a copy; the next tile's page ids are on their way while this one's copies go out.  A warp issues a copy in
    // 30 ns: where a chunk is 8 or 16 of them (pages of 16 and 8 rows) two warps share the chunks.  16 requests of 32k
    // tokens with 96 heads: pages of 8 148.5 us by one warp, 97.6 by two; of 16 99.5 and 95.7; of 64 95.5.
    if (lane == 0) prefetch_tmap(&tmap_kv);
    int32_t rho = box_row(a, w, lane), page = page_of(a, w, rho);
    Slots slots = slots_of(kKeysHeld);
    if (kQ4) slots.empty = &bars[kRFree];
    bool ok = true, more = true;
    while (more && ok) {
      const int32_t y = pool_row(a, w.rs, rho, page);
      if (kKeysHeld) w.g = w.g1 - 1;  // the groups between meet the same keys
      more = w.next(a, rank);
      rho = more ? box_row(a, w, lane) : -1;
      page = page_of(a, w, rho);
      const uint32_t who = __ballot_sync(0xffffffffu, y >= 0);
      if (kQ4) {
        ok = slots.wait(abort_s);
        if (!ok) break;
        uint64_t* full = &bars[kRFull + slots.at];
        if (lane == 0) mbar_arrive_expect_tx(full, __popc(who) * a.box_rows * kQ4RowBytes);
        __syncwarp();
        if (y >= 0)
          bulk_load(smem + sl.ring + slots.at * kRawTile + lane * a.box_rows * kQ4RowBytes,
                    a.arena + (int64_t)y * kQ4RowBytes, a.box_rows * kQ4RowBytes, full);
        slots.advance();
      } else {
        for (int c = 0; c < kChunks && ok; ++c) {
          if (two && (slots.uses & 1) != (warp == kKeyWarp2)) {
            slots.advance();
            continue;
          }
          ok = slots.wait(abort_s);
          if (!ok) break;
          if (lane == 0) expect_tx_cluster(slots.full_bar(), __popc(who) * a.box_rows * 128);
          __syncwarp();
          if (y >= 0)
            tma_load_2d_pair(slots.dst() + lane * a.box_rows * 128, &tmap_kv, slots.full_bar(), c * kChunkDims, y);
          slots.advance();
        }
      }
    }
    if (ok) slots.drain(abort_s);
  } else if (warp == kQueryWarp && any) {
    // ------------------------------------------------------------------ queries in
    if (lane == 0) prefetch_tmap(&tmap_q);
    Slots slots = slots_of(!kKeysHeld);
    bool ok = true, more = true;
    while (more && ok) {
      if (w.group_begins()) {
        const int32_t y = w.b * a.R + w.g * a.Rg + rank * (a.Rg / 2);
        for (int c = 0; c < kChunks && ok; ++c) {
          ok = slots.wait(abort_s);
          if (!ok) break;
          if (lane == 0) {
            expect_tx_cluster(slots.full_bar(), a.Rg / 2 * 128);
            tma_load_2d_pair(slots.dst(), &tmap_q, slots.full_bar(), c * kChunkDims, y);
          }
          slots.advance();
        }
      }
      more = w.next(a, rank);
    }
    if (ok) slots.drain(abort_s);
  } else if (warp == kMmaWarp && any && rank == 0) {
    // ------------------------------------------------------------------ products (the leader's alone)
    // The whole warp walks and waits, one lane issues: the operands' descriptors are then uniform values.  (With one
    // lane in a loop of its own each product's came through vector registers, 760 cycles a chunk in all.)
    const bool one = elect_one();
    const uint32_t idesc = idesc_bf16_f32(2 * kKeys, a.Rg, 0, 0);
    const uint64_t held0 = sw128_desc(smem_u32(smem) + sl.held, 16, 1024);
    const uint64_t ring0 = sw128_desc(smem_u32(smem) + sl.ring, 16, 1024);
    const uint32_t held_step = (uint32_t)a.held_bytes >> 4, ring_step = (uint32_t)a.ring_bytes >> 4;
    const uint32_t slots = kQ4 ? kASlots : a.stages;
    uint32_t st = 0, ph = 0, hph = 0, j = 0;
    bool ok = true, more = true;
    while (more && ok) {
      const bool first = w.first<kKeysHeld>(), last = w.last<kKeysHeld>();
      const uint32_t buf = j & 1, d = tmem + (kQ4 ? 128 : 256) * buf;
      ok = sleep_wait(&bars[kSFree + buf], ((j >> 1) & 1) ^ 1, abort_s);
      for (int c = 0; c < (kQ4 ? kAParts : kChunks) && ok; ++c) {
        const int h0 = kQ4 ? 2 * c : c, nh = kQ4 && c < kAParts - 1 ? 2 : 1;  // held chunks of this step
        if (first)
          for (int i = 0; i < nh; ++i) ok = ok && sleep_wait(&bars[kHeldFull + h0 + i], hph, abort_s);
        ok = ok && sleep_wait(&bars[(kQ4 ? kAFull : kFull) + st], ph, abort_s);
        if (!ok) break;
        tc_fence_after();
        const uint64_t hd = held0 + h0 * held_step, rd = ring0 + st * ring_step;
        const uint64_t qd = kKeysHeld ? rd : hd, kd = kKeysHeld ? hd : rd;
        const uint32_t kt = tmem + kACol + 64 * st;
        if (one) {
#pragma unroll
          for (int k = 0; k < kChunkDims / 16; ++k) {
            if (kQ4)
              mma_pair_ts(d, kt + 8 * k, hd + 2 * k, idesc, (c | k) != 0);
            else
              mma_pair_ss(d, kd + 2 * k, qd + 2 * k, idesc, (c | k) != 0);
          }
          if (kQ4 && nh == 2) {
#pragma unroll
            for (int k = 0; k < kChunkDims / 16; ++k) mma_pair_ts(d, kt + 32 + 8 * k, hd + held_step + 2 * k, idesc, 1);
          }
          commit_pair(&bars[(kQ4 ? kAEmpty : kEmpty) + st]);
          if (last)
            for (int i = 0; i < nh; ++i) commit_pair(&bars[kHeldEmpty + h0 + i]);
          if (h0 == kChunks - 1) commit_pair(&bars[kSFull + buf]);
        }
        __syncwarp();
        if (++st == slots) {
          st = 0;
          ph ^= 1;
        }
      }
      if (!ok) break;
      if (first) hph ^= 1;
      ++j;
      more = w.next(a, rank);
    }
  } else if (warp < 4 && any) {
    // ------------------------------------------------------------------ sums: a thread a key
    // What a tile wants from global memory (its key's page and old weight) is loaded while the tile before is summed.
    const float c = a.scale_log2;
    const uint64_t c2 = f2_pack(__float_as_uint(c), __float_as_uint(c));
    struct Key {
      int64_t at;         // its entry of weights, -1: not written
      float old;
      int32_t page, col0; // first column of the group that sees it
      int32_t ncols, i;   // columns of the group, pair-tile of the block
      int64_t lse_at;     // the group's first row, -1: as before
      bool add;           // to the groups' sum so far
      bool joins;         // the tile's last group here, and another pair has begun it
    };
    const bool keeps = a.old_lens && a.decay != 0.f;
    int32_t old_b = -1;
    int64_t old_len = 0;
    auto look = [&]() -> Key {
      Key k;
      k.ncols = min(a.Rg, a.R - w.g * a.Rg);
      k.i = w.i;
      k.lse_at = w.group_begins() ? (int64_t)w.b * a.R + w.g * a.Rg : -1;
      k.add = w.g > w.g0;
      k.joins = w.g0 > 0 && w.g == w.g1 - 1;
      k.at = -1;
      k.old = 0.f;
      k.page = k.col0 = 0;
      if (keeps && w.b != old_b) {
        old_b = w.b;
        old_len = __ldg(a.old_lens + w.b);
      }
      const int32_t row = w.t * kKeys + warp * 32 + lane;
      if (row < w.rows) {
        const int32_t I = (int32_t)a.L.I, blk = I == 1 ? row : row / I;
        const int64_t p = ((int64_t)blk * a.L.N + a.shard_begin + w.rs) * I + (row - blk * I);
        const int64_t hidden = p - (w.sh.S - a.q_len);  // query tokens [0, hidden) come before this key
        if (hidden > 0) {
          const int64_t x = hidden * a.H - (int64_t)w.g * a.Rg;
          k.col0 = (int32_t)(x < 0 ? 0 : (x > a.Rg ? a.Rg : x));
        }
        if (w.g == w.g1 - 1) {
          k.page = __ldg(a.bt + (int64_t)w.b * a.bt_stride + row / (int32_t)a.L.P);
          k.at = ((int64_t)w.rs * a.B + w.b) * a.w_stride + row;
          if (keeps && p < old_len && w.g0 == 0) k.old = a.weights[k.at];
        }
      }
      return k;
    };
    bool ok = true, more = true;
    uint32_t j = 0;
    float part = 0.f;  // a tile's sum over the groups so far (4-bit: in acc_s, by tile of the block)
    Key key = look();
    while (more && ok) {
      const Key now = key;
      float l[8];
      if (now.lse_at >= 0) {
#pragma unroll
        for (int k = 0; k < 8; ++k) l[k] = lane + 32 * k < now.ncols ? __ldg(a.lse + now.lse_at + lane + 32 * k) : 0.f;
      }
      more = w.next(a, rank);
      if (more) key = look();
      const uint32_t buf = j & 1;
      ok = sleep_wait(&bars[kSFull + buf], (j >> 1) & 1, abort_s);
      if (!ok) break;
      tc_fence_after();
      if (now.lse_at >= 0) {
        // A new group's columns, in the buffer of the group before last: this tile's scores are there, so every warp has
        // freed those of the tile before last, and with them that group.  All warps write the same values.
        lse_s = reinterpret_cast<float*>(smem + sl.lse) + (lse_s == reinterpret_cast<float*>(smem + sl.lse) ? 256 : 0);
#pragma unroll
        for (int k = 0; k < 8; ++k)  // a row that saw nothing adds 2^-inf
          lse_s[lane + 32 * k] = l[k] == -INFINITY ? -INFINITY : -(a.base2 ? l[k] : l[k] * kLog2e);
        __syncwarp();
      }
      const uint32_t s_addr = tmem + ((uint32_t)(warp * 32) << 16) + (kQ4 ? 128 : 256) * buf;
      // Some key of the warp is hidden from some rows: its exponentials are cleared by a bit mask, and blocks that see
      // none are left out.  (Comparing every column with the key's first took longer than the products of a tile, and with
      // it the pairs that have a request's last keys: the 64-token window 260 us against 237.)
      const bool hides = __any_sync(0xffffffffu, now.col0 > 0);
      uint64_t sum[2] = {0, 0};
      for (int k0 = 0; k0 < now.ncols; k0 += 32) {
        uint32_t vis = ~0u;  // columns [k0, k0 + 32) that count for this key: a bit each
        uint32_t r[32];
        auto add = [&](bool masked) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float4 l = *reinterpret_cast<const float4*>(lse_s + k0 + 4 * k);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint64_t x = f2_fma(f2_pack(r[4 * k + 2 * e], r[4 * k + 2 * e + 1]), c2,
                                        f2_pack(__float_as_uint(e ? l.z : l.x), __float_as_uint(e ? l.w : l.y)));
              uint32_t x0, x1;
              f2_unpack(x, x0, x1);
              float e0 = fast_exp2(__uint_as_float(x0)), e1 = fast_exp2(__uint_as_float(x1));
              if (masked) {  // after the exponential: a hidden row's NaN does not count
                e0 = vis >> (4 * k + 2 * e) & 1 ? e0 : 0.f;
                e1 = vis >> (4 * k + 2 * e + 1) & 1 ? e1 : 0.f;
              }
              sum[e] = f2_add(sum[e], f2_pack(__float_as_uint(e0), __float_as_uint(e1)));
            }
          }
        };
        if (!hides && k0 + 32 <= now.ncols) {
          tmem_ld32_sync(s_addr + k0, r);
          add(false);
          continue;
        }
        vis = now.col0 <= k0 ? ~0u : now.col0 >= k0 + 32 ? 0u : ~0u << (now.col0 - k0);
        if (now.ncols < k0 + 32) vis &= (1u << (now.ncols - k0)) - 1;
        if (!__any_sync(0xffffffffu, vis)) continue;
        tmem_ld32_sync(s_addr + k0, r);
        add(true);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_cluster(lead + 8 * (kSFree + buf));
      uint32_t x0, x1;
      f2_unpack(f2_add(sum[0], sum[1]), x0, x1);
      float s = __uint_as_float(x0) + __uint_as_float(x1);
      if (a.ngroups > 1) {
        float* acc = kQ4 ? acc_s + now.i * kKeys + warp * 32 + lane : &part;  // this thread's own
        if (now.add) s += *acc;
        *acc = s;
      }
      const bool there = now.at >= 0 && now.page >= 0 && now.page < a.pool_pages;
      if (now.joins) {
        const int32_t k = pair * 2 * kKeys + rank * kKeys + warp * 32 + lane;
        a.part_at[k] = there ? now.at : -1;
        a.part[k] = s;
      } else if (there) {
        a.weights[now.at] = (now.old == INFINITY ? 0.f : a.decay * now.old) + s;  // +inf: marked as having none
      }
      ++j;
    }
  } else if (kQ4 && warp >= kDequantWarp && any) {
    // ------------------------------------------------------------------ 4-bit rows -> operands in TMEM
    // Warp 8 + 4 s + k: keys [32 k, 32 k + 32) of every kDequantSets-th slot.  Every pair-tile of the run is met
    // once a row group; a CTA without a tile in the last of a request turns over what its slot holds, for nobody.
    const int set = (warp - kDequantWarp) >> 2, quarter = warp & 3;
    const uint32_t lane_addr = tmem + ((uint32_t)(quarter * 32) << 16) + kACol;
    const uint32_t tiles = (uint32_t)start_s[5];
    uint32_t rb = 0, rph = 0;  // raw tile and its parity
    bool ok = true;
    for (uint32_t j = 0; j < tiles && ok; ++j) {
      ok = sleep_wait(&bars[kRFull + rb], rph, abort_s);
      const uint32_t row_s = smem_u32(smem) + sl.ring + rb * kRawTile + (quarter * 32 + lane) * kQ4RowBytes;
      for (int part = 0; part < kAParts && ok; ++part) {
        const uint32_t n = j * kAParts + part, slot = n % kASlots;
        if (n % kDequantSets != (uint32_t)set) continue;
        const uint32_t to = lane_addr + 64 * slot;
        uint32_t v[32];
        if (part < kAParts - 1) {
          uint32_t c0[8], c1[8], s0, s1;
          load32(row_s + 64 * part, c0);
          load32(row_s + 64 * part + 32, c1);
          asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(s0), "=r"(s1) : "r"(row_s + kQ4ScaleOff + 8 * part));
          ok = sleep_wait(&bars[kAEmpty + slot], ((n / kASlots) & 1) ^ 1, abort_s);
          if (!ok) break;
          tc_fence_after();
          dequant_chunk(c0, s0, v);
          tmem_st32(to, v);
          dequant_chunk(c1, s1, v);
          tmem_st32(to + 32, v);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) load32(row_s + kQ4RopeOff + 32 * k, v + 8 * k);
          ok = sleep_wait(&bars[kAEmpty + slot], ((n / kASlots) & 1) ^ 1, abort_s);
          if (!ok) break;
          tc_fence_after();
          tmem_st32(to, v);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_cluster(lead + 8 * (kAFull + slot));
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kRFree + rb]);
      if (++rb == (uint32_t)a.stages) {
        rb = 0;
        rph ^= 1;
      }
    }
    // the operand slots' last releases land before the CTA may leave
    const uint32_t n = tiles * kAParts;
    for (uint32_t s = 0; s < kASlots && s < n && ok; ++s) {
      const uint32_t uses = (n - 1 - s) / kASlots;
      ok = sleep_wait(&bars[kAEmpty + s], uses & 1, abort_s);
    }
  }
  __syncthreads();
  if (*abort_s) {
    if (tid == 0) flag(a.status, DCP_STATUS_TIMEOUT);
    const uint64_t t0 = globaltimer();  // copies and products in flight land before memory is given back
    while (globaltimer() - t0 < 100000) {
    }
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kAllCols) : "memory");
}

// What the pairs after the first have of a tile that several share, added to what the first has written: a block a
// boundary between two runs, a thread a key, the pairs in order.
__global__ void __launch_bounds__(2 * kKeys) join_kernel(WeighArgs a) {
  const int p = blockIdx.x + 1;
  const int64_t units = *a.units;  // 0: nothing is shared
  const int64_t u = run_start(units, p, a.npairs), tile = u - u % a.ngroups;
  if (u == tile || run_start(units, p - 1, a.npairs) > tile) return;  // not the first boundary within a tile
  int64_t at = -1, k0 = u;
  float s = 0.f;
  for (int k = p; k < a.npairs && k0 < tile + a.ngroups; ++k) {
    const int64_t k1 = run_start(units, k + 1, a.npairs);
    if (k1 > k0) {
      at = a.part_at[k * 2 * kKeys + threadIdx.x];
      s += a.part[k * 2 * kKeys + threadIdx.x];
    }
    k0 = k1;
  }
  if (at >= 0 && at < a.w_stride * a.B * a.n_held) a.weights[at] += s;  // (after a timeout it may be anything)
}

constexpr int kMaxPairs = 128;
// Tiles are shared from this many row groups on.  A whole tile is then 15 us of a pair's products and more; the second
// launch and its scratch cost 3 us, 10 on the host.
constexpr int kShareGroups = 4;
constexpr size_t kUnitsBytes = 128, kPartAtBytes = (size_t)kMaxPairs * 2 * kKeys * sizeof(int64_t),
                 kPartBytes = (size_t)kMaxPairs * 2 * kKeys * sizeof(float);
size_t workspace_size(int64_t R, bool q4) {
  return R > kShareGroups * (q4 ? 128 : 256) ? kUnitsBytes + kPartAtBytes + kPartBytes : 0;
}

PairKernel g_bf16(reinterpret_cast<const void*>(&weigh_kernel<false, false>), kThreads);
PairKernel g_bf16_groups(reinterpret_cast<const void*>(&weigh_kernel<false, true>), kThreads);
PairKernel g_q4(reinterpret_cast<const void*>(&weigh_kernel<true, false>), kThreadsQ4);

struct WeighCall {
  const dcp_layout_t* layout;
  int32_t shard_begin, shard_end;
  const void* q;
  int32_t B, q_len, H;
  const void* arena;
  int64_t pool_pages;
  const int32_t* block_table;
  int64_t bt_stride, max_pages;
  const int64_t* seq_lens;
  float scale;
  int32_t lse_base;
  const float* lse;
  const int64_t* old_lens;
  float decay;
  float* weights;
  int64_t w_stride;
  void* workspace;
  size_t workspace_bytes;
  int32_t* status;
  void* stream;
};

template <bool kQ4>
int32_t weigh(const WeighCall& c) {
  // the partial decode's checks, with the weights in the place of its outputs
  const DecodeCall d{c.layout, c.shard_begin, c.shard_end, c.q, c.B, c.q_len, c.H, c.arena, c.pool_pages,
                     c.block_table, c.bt_stride, c.max_pages, c.seq_lens, c.scale, c.lse_base, c.arena ? const_cast<void*>(c.arena) : nullptr,
                     DCP_F32, c.weights, c.status, c.stream};
  const int32_t rc = check_decode_args(d);
  if (rc != DCP_OK) return rc;
  if (!c.lse || !(c.decay >= 0.f) || !(c.decay < INFINITY) || c.w_stride / c.layout->page_size < c.max_pages)
    return DCP_ERR_INVALID;
  if ((uintptr_t)c.workspace % 16 != 0) return DCP_ERR_INVALID;
  if (c.workspace && c.workspace_bytes < workspace_size((int64_t)c.q_len * c.H, kQ4)) return DCP_ERR_WORKSPACE;
  WeighArgs a;
  a.L = to_layout(c.layout);
  a.shard_begin = c.shard_begin;
  a.n_held = c.shard_end - c.shard_begin;
  a.B = c.B;
  a.q_len = c.q_len;
  a.H = c.H;
  a.R = c.q_len * c.H;
  // groups of at most 256 (128) rows, as equal as multiples of 32 allow (half of them in each CTA)
  const int most = kQ4 ? 128 : 256;
  const int groups = (a.R + most - 1) / most;
  a.Rg = ((a.R + groups - 1) / groups + 31) / 32 * 32;
  a.ngroups = (a.R + a.Rg - 1) / a.Rg;
  const bool keys_held = !kQ4 && a.ngroups > 1;
  const int q_chunk = a.Rg / 2 * 128;
  a.held_bytes = keys_held ? kStageBytes : q_chunk;
  a.ring_bytes = kQ4 ? kRawTile : keys_held ? q_chunk : kStageBytes;
  a.stages = (int32_t)(kSmemBudget - smem_of(a.held_bytes, 0, 0, kQ4).total) / a.ring_bytes;
  a.stages = std::min(a.stages, kQ4 ? kMaxRaw : kMaxStages);
  const size_t smem = smem_of(a.held_bytes, a.stages, a.ring_bytes, kQ4).total;
  a.block = kQ4 ? kBlockQ4 : 1;
  a.box_rows = std::min(c.layout->page_size, kTile);
  a.nbox = kKeys / a.box_rows;
  PairKernel& kernel = kQ4 ? g_q4 : keys_held ? g_bf16_groups : g_bf16;
  a.npairs = std::min(kernel.max_active_clusters(kSmemBudget), kMaxPairs);  // one CTA an SM, whatever the sizes are
  if (a.npairs < 1) return DCP_ERR_CUDA;
  a.pool_pages = c.pool_pages;
  a.pool_rows = c.pool_pages * c.layout->page_size;
  a.max_rows = table_rows(c.layout, c.max_pages);
  a.arena = static_cast<const unsigned char*>(c.arena);
  a.bt = c.block_table;
  a.bt_stride = c.bt_stride;
  a.max_pages = c.max_pages;
  a.seq_lens = c.seq_lens;
  a.scale_log2 = kQ4 ? c.scale * kLog2e : (float)((double)c.scale * 1.4426950408889634 * (1.0 + kTruncation));
  a.base2 = c.lse_base == DCP_LSE_BASE_2;
  a.lse = c.lse;
  a.old_lens = c.old_lens;
  a.decay = c.decay;
  a.weights = c.weights;
  a.w_stride = c.w_stride;
  a.status = c.status;
  unsigned char* ws = workspace_size(a.R, kQ4) > 0 ? static_cast<unsigned char*>(c.workspace) : nullptr;
  a.units = reinterpret_cast<int64_t*>(ws);
  a.part_at = reinterpret_cast<int64_t*>(ws ? ws + kUnitsBytes : nullptr);
  a.part = reinterpret_cast<float*>(ws ? ws + kUnitsBytes + kPartAtBytes : nullptr);
  CUtensorMap tq, tkv;
  if (!make_tmap(&tq, c.q, (uint64_t)c.B * a.R, (uint32_t)a.Rg / 2)) return DCP_ERR_CUDA;
  if (kQ4)
    tkv = tq;  // its rows are copied as they are
  else if (!make_tmap(&tkv, c.arena, (uint64_t)a.n_held * a.pool_rows, (uint32_t)a.box_rows))
    return DCP_ERR_CUDA;
  if (!kernel.ensure_smem(kSmemBudget)) return DCP_ERR_CUDA;
  const auto run = kQ4 ? weigh_kernel<true, false> : keys_held ? weigh_kernel<false, true> : weigh_kernel<false, false>;
  run<<<2 * a.npairs, kQ4 ? kThreadsQ4 : kThreads, smem, as_stream(c.stream)>>>(tq, tkv, a);
  if (!ws || a.npairs == 1) return launch_status();
  join_kernel<<<a.npairs - 1, 2 * kKeys, 0, as_stream(c.stream)>>>(a);
  return launch_status(2);
}

}  // namespace

extern "C" int32_t dcp_mla_key_weights(const dcp_layout_t* layout, int32_t shard_begin, int32_t shard_end, const void* q,
                                       int32_t B, int32_t q_len, int32_t H, const void* arena, int64_t pool_pages,
                                       const int32_t* block_table, int64_t bt_stride, int64_t max_pages,
                                       const int64_t* seq_lens, float scale, int32_t lse_base, const float* lse,
                                       const int64_t* old_lens, float decay, float* weights, int64_t w_stride,
                                       void* workspace, size_t workspace_bytes, int32_t* status, void* stream) {
  return weigh<false>(WeighCall{layout, shard_begin, shard_end, q, B, q_len, H, arena, pool_pages, block_table, bt_stride,
                                max_pages, seq_lens, scale, lse_base, lse, old_lens, decay, weights, w_stride, workspace,
                                workspace_bytes, status, stream});
}

extern "C" int32_t dcp_mla_key_weights_q4(const dcp_layout_t* layout, int32_t shard_begin, int32_t shard_end,
                                          const void* q, int32_t B, int32_t q_len, int32_t H, const void* arena,
                                          int64_t pool_pages, const int32_t* block_table, int64_t bt_stride,
                                          int64_t max_pages, const int64_t* seq_lens, float scale, int32_t lse_base,
                                          const float* lse, const int64_t* old_lens, float decay, float* weights,
                                          int64_t w_stride, void* workspace, size_t workspace_bytes, int32_t* status,
                                          void* stream) {
  return weigh<true>(WeighCall{layout, shard_begin, shard_end, q, B, q_len, H, arena, pool_pages, block_table, bt_stride,
                               max_pages, seq_lens, scale, lse_base, lse, old_lens, decay, weights, w_stride, workspace,
                               workspace_bytes, status, stream});
}

extern "C" size_t dcp_mla_key_weights_workspace_size(int32_t q_len, int32_t H) {
  return q_len > 0 && H > 0 ? workspace_size((int64_t)q_len * H, false) : 0;
}

extern "C" size_t dcp_mla_key_weights_workspace_size_q4(int32_t q_len, int32_t H) {
  return q_len > 0 && H > 0 ? workspace_size((int64_t)q_len * H, true) : 0;
}
