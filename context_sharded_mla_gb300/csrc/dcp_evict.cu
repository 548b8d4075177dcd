// dcp_evict.cu — a cache made shorter by what its rows weigh: which rows of each shard
// stay, and their move to the front of the shard, in place.
//
// Each shard keeps count_r(new length) of its own rows ("PCP / DCP：计算、KV 布局与块
// 轮转", section 6: local_len), so that no row leaves its shard and the layout's count
// rule holds for what is left; kept rows stay in order.
//
// select_kernel: one cluster of CTAs for a (request, shard) unit, each thread holding its
// rows' weights in registers as integers of the same order.  The k-th largest of the rows
// that compete is found digit by digit: 12 bits first (one histogram a CTA; weights of one
// magnitude share their first bits, but few lanes of a warp the first 12), the others among
// the keys of that bin alone.  Rows are then written in order: ballots, and a sum over the
// warps.  Only whole numbers are added, so the result depends on no order.  Bound by
// latency: two CTAs an SM go from load to histogram to scan to list to write, a block
// barrier between each, with no load of a next unit under way (53 % of the issue slots, 13 %
// of DRAM).  512 units of 16384 rows (33 MB) take 28 us, 1.2 TB/s; a unit of a few rows 5 us.
//
// mark_kernel: rows that no query has weighed get the weight +infinity, which the
// selection keeps before any other number and the next weights take for none.  A launch and
// two loads: 8 rows of 64 requests on 8 shards 2.2 us, all 16384 of each 6.3.
//
// compact_kernel: row i <- row kept[i] >= i.  Writing row i is safe once the rows up to
// i have been read: a later row j > i reads kept[j] >= j.  So a cluster walks a unit in
// windows, reads a window (bulk copies into a ring of slots in shared memory, several
// windows ahead), and writes it when every CTA of the cluster has its part of it.
// Memory-bound: 2 * 1152 (or 416) bytes a row; 524288 rows in 194 us, 6.3 TB/s (4-bit: 236
// us with their read-back).
#include <algorithm>

#include "dcp_internal.cuh"

#include "sm100_ptx.cuh"

using namespace dcp;
using namespace dcp::sm100;

namespace {

// ---------------------------------------------------------------- select
constexpr int kSelThreads = 512, kSelWarps = kSelThreads / 32, kDigits = 4, kBins = 256;

struct SelectArgs {
  Layout L;
  int32_t shard_begin, n_held, B;
  const int64_t *seq_lens, *new_lens;
  int64_t sinks, recent;
  const float* weights;
  int64_t w_stride;
  int32_t* kept;
  int64_t kept_stride;
  int32_t* status;
};

// Unsigned integers in the order of the weights; a NaN above all, -0 as 0.
__device__ __forceinline__ uint32_t order_key(float w) {
  const uint32_t u = __float_as_uint(__fadd_rn(w, 0.f));  // -0 becomes 0, a NaN 0x7fffffff
  return w != w ? 0xFFFFFFFFu : u ^ (0x80000000u | (uint32_t)((int32_t)u >> 31));
}

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ uint32_t cluster_nctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ int warp_sum(int v) {
#pragma unroll
  for (int s = 16; s; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  return v;
}

// A unit's parts: rows [0, lo) are sinks, [hi, n) recent ones, those between compete for `want` places.
struct Unit {
  int32_t lo, hi, ns;
  uint32_t want;
};

// Rows of shard r below position x (32-bit division where it does: a 64-bit one is some hundred instructions).
__device__ __forceinline__ int64_t rows_below(int64_t r, int64_t x, const Layout& L) {
  const int64_t blk = L.N * L.I;
  const int64_t k = ((x | blk) >> 31) == 0 ? (int64_t)((uint32_t)x / (uint32_t)blk) : x / blk;
  int64_t rem = x - k * blk - r * L.I;
  rem = rem < 0 ? 0 : (rem > L.I ? L.I : rem);
  return k * L.I + rem;
}

// Sets u up and writes its sinks and recent rows; false (for the whole cluster) where no row competes, or the unit is
// refused.
__device__ bool select_begin(const SelectArgs& a, int64_t unit, uint32_t rank, uint32_t nranks, Unit* u) {
  const int rs = (int)(unit / a.B), b = (int)(unit % a.B), tid = threadIdx.x;
  const int64_t S = a.seq_lens[b], M = a.new_lens[b], r = a.shard_begin + rs;
  const int64_t m = M > 0 ? rows_below(r, M, a.L) : 0, n = S > 0 ? rows_below(r, S, a.L) : 0;
  int32_t* kept = a.kept + unit * a.kept_stride;
  if (M < 0 || M > S || n > a.w_stride || m > a.kept_stride) {
    if (tid == 0 && rank == 0) flag(a.status, DCP_STATUS_BAD_LENGTH);
    const int64_t e = m < a.kept_stride ? m : a.kept_stride;
    for (int64_t i = rank * kSelThreads + tid; i < e; i += nranks * kSelThreads) kept[i] = -1;
    return false;
  }
  const int64_t lo = rows_below(r, a.sinks < S ? a.sinks : S, a.L);
  const int64_t zr = rows_below(r, S > a.recent ? S - a.recent : 0, a.L);
  const int64_t hi = zr > lo ? zr : lo, ns = lo < m ? lo : m, nr = m - ns < n - hi ? m - ns : n - hi;
  u->lo = (int32_t)lo;  // rows of a unit fit 31 bits (w_stride)
  u->hi = (int32_t)hi;
  u->ns = (int32_t)ns;
  u->want = (uint32_t)(m - ns - nr);
  if (rank == 0)
    for (int64_t i = tid; i < ns; i += kSelThreads) kept[i] = (int32_t)i;
  if (rank == nranks - 1)
    for (int64_t i = tid; i < nr; i += kSelThreads) kept[m - nr + i] = (int32_t)(n - nr + i);
  return u->want != 0;
}

constexpr int kCopies = 16;                 // of a histogram of 256 bins: lanes l and l + 16 share one
constexpr int kTopBits = 12, kTopBins = 1 << kTopBits;  // first digit of the keys in registers: one copy of 4096 bins
constexpr int kFewKeys = 2048;              // candidates that get a list of their own
struct SelectSmem {
  uint32_t hist[kBins * kCopies];    // or [kTopBins]
  uint32_t total[kDigits][kBins];    // this CTA's counts of each digit's bins, read by the cluster
  uint32_t all[kBins];
  uint32_t pick[3];                  // chosen bin, rows still wanted of it, rows in it
  uint32_t cta_n[2];                 // rows above and at the limit
};
static_assert(kTopBins == kBins * kCopies, "one buffer for both");

__device__ __forceinline__ void clear_hist(SelectSmem& sm) {
  for (int i = threadIdx.x; i < kTopBins / 4; i += kSelThreads) reinterpret_cast<uint4*>(sm.hist)[i] = make_uint4(0, 0, 0, 0);
  __syncthreads();
}

__device__ __forceinline__ void count_digit(SelectSmem& sm, uint32_t digit) {
  atomicAdd(&sm.hist[digit * kCopies + (threadIdx.x & (kCopies - 1))], 1u);
}

// After a digit's histogram: the bin that holds the want-th largest of the cluster's candidates.
__device__ void choose_bin(SelectSmem& sm, int d, uint32_t want, uint32_t nranks) {
  const int tid = threadIdx.x, lane = tid & 31;
  __syncthreads();
  if (tid < kBins) {
    uint32_t s = 0;
#pragma unroll
    for (int k = 0; k < kCopies; ++k) s += sm.hist[tid * kCopies + ((k + tid) & (kCopies - 1))];
    sm.total[d][tid] = s;
  }
  if (nranks > 1) {
    cluster_sync();
    if (tid < kBins) {
      uint32_t s = 0;
      for (uint32_t c = 0; c < nranks; ++c) s += ld_cluster_u32(mapa_shared(smem_u32(&sm.total[d][tid]), c));
      sm.all[tid] = s;
    }
  }
  __syncthreads();
  if (tid < 32) {  // counts from the top, 8 bins a lane
    const uint32_t* all = nranks > 1 ? sm.all : sm.total[d];
    uint32_t c[8], s = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) s += c[k] = all[255 - 8 * lane - k];
    uint32_t incl = s;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, incl, x);
      if (lane >= x) incl += y;
    }
    uint32_t before = incl - s;
    if (before < want && want <= incl) {  // exactly one lane
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (before < want && want <= before + c[k]) {
          sm.pick[0] = 255 - 8 * lane - k;
          sm.pick[1] = want - before;
          sm.pick[2] = c[k];
        }
        before += c[k];
      }
    }
  }
  __syncthreads();
}

// The same for the first digit of the keys in registers, 4096 bins.  In a cluster every CTA adds up an equal part of the
// bins over all of them (each reading all 4096 bins of all took 40000 clocks with 8 CTAs, distributed shared memory giving
// some 3 bytes a clock), then all look through the part that holds the bin.  `sums`: room for kTopBins / 2 of them.
__device__ void choose_top(SelectSmem& sm, uint32_t* sums, uint32_t* warp_s, uint32_t want, uint32_t rank,
                           uint32_t nranks) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t part = kTopBins / nranks;  // nranks is a power of two
  uint32_t first = 0, from = smem_u32(sm.hist);
  if (nranks > 1) {
    if (tid == 0) sm.cta_n[1] = 0;
    cluster_sync();
    uint32_t mine = 0;
    for (uint32_t i = tid; i < part; i += kSelThreads) {
      uint32_t s = 0;
#pragma unroll 8
      for (uint32_t r = 0; r < nranks; ++r) s += ld_cluster_u32(mapa_shared(smem_u32(sm.hist + rank * part + i), r));
      sums[i] = s;
      mine += s;
    }
    mine = warp_sum(mine);
    if (lane == 0) atomicAdd(&sm.cta_n[1], mine);
    cluster_sync();
    uint32_t r = nranks, n = 0;
    do {  // parts from the top, until the one that holds the want-th
      want -= n;
      --r;
      n = ld_cluster_u32(mapa_shared(smem_u32(&sm.cta_n[1]), r));
    } while (n < want && r > 0);
    first = r * part;
    from = mapa_shared(smem_u32(sums), r);
  } else {
    __syncthreads();
  }
  // part / 512 bins a thread, from the top
  const uint32_t per = part / kSelThreads, at = part - per * (tid + 1);
  uint32_t c[8], s = 0;
  if (nranks > 1) {
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k) c[k] = k < per ? ld_cluster_u32(from + 4 * (at + k)) : 0;
  } else {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint4 x = ld_shared_v4(from + 4 * at + 16 * k);
      c[4 * k] = x.x; c[4 * k + 1] = x.y; c[4 * k + 2] = x.z; c[4 * k + 3] = x.w;
    }
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) s += c[k];
  uint32_t incl = s;
#pragma unroll
  for (int x = 1; x < 32; x <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, incl, x);
    if (lane >= x) incl += y;
  }
  if (lane == 31) warp_s[warp] = incl;
  if (nranks > 1) cluster_sync(); else __syncthreads();  // and every count has been read
  uint32_t before = incl - s;
  for (int i = 0; i < warp; ++i) before += warp_s[i];
  if (before < want && want <= before + s) {  // exactly one thread
#pragma unroll
    for (int k = 7; k >= 0; --k) {
      if (before < want && want <= before + c[k]) {
        sm.pick[0] = first + at + k;
        sm.pick[1] = want - before;
        sm.pick[2] = c[k];
      }
      before += c[k];
    }
  }
  __syncthreads();
}

// Units of at most kPer * 512 rows a CTA: every thread holds its kPer keys in registers (warp w has rows
// [32 kPer w, 32 kPer (w + 1)) of the CTA's, lane by lane; key 0, which is no weight's and lies below all, where there
// is none), so that the weights are read once.  Few keys share a first digit of 12 bits: those of the chosen bin go to
// a list, and the other digits are looked for there.
template <int kPer>
__global__ void __launch_bounds__(kSelThreads, 2) select_kernel(SelectArgs a) {
  __shared__ __align__(16) SelectSmem sm;
  __shared__ uint32_t few[kFewKeys];
  __shared__ uint32_t warp_s[kSelWarps];  // rows at (<< 16) and above the limit (at most 16384: the halves do not meet)
  const uint32_t rank = cluster_ctarank(), nranks = cluster_nctarank();
  const int64_t unit = blockIdx.x / nranks;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Unit u;
  if (!select_begin(a, unit, rank, nranks, &u)) return;
  const int32_t len = u.hi - u.lo, per = (len + nranks - 1) / nranks;
  const int32_t c1 = min((int32_t)(rank + 1) * per, len);
  const int32_t i0 = min((int32_t)rank * per, len) + warp * (32 * kPer) + lane;
  const float* w = a.weights + unit * a.w_stride + u.lo + i0;
  uint32_t key[kPer];
  const bool whole = i0 - lane + 32 * kPer <= c1;  // uniform over the warp
  if (whole) {
#pragma unroll
    for (int k = 0; k < kPer; ++k) key[k] = __float_as_uint(__ldg(w + 32 * k));
  } else {
#pragma unroll
    for (int k = 0; k < kPer; ++k) key[k] = i0 + 32 * k < c1 ? __float_as_uint(__ldg(w + 32 * k)) : 0u;
  }
  clear_hist(sm);
  if (tid == 0) sm.cta_n[0] = 0;
  if (whole) {
#pragma unroll
    for (int k = 0; k < kPer; ++k) key[k] = order_key(__uint_as_float(key[k]));
  } else {
#pragma unroll
    for (int k = 0; k < kPer; ++k) key[k] = i0 + 32 * k < c1 ? order_key(__uint_as_float(key[k])) : 0u;
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k) atomicAdd(&sm.hist[key[k] >> (32 - kTopBits)], 1u);
  uint32_t want = u.want;
  choose_top(sm, few, warp_s, want, rank, nranks);
  uint32_t limit = sm.pick[0] << (32 - kTopBits);
  want = sm.pick[1];
  if (want < sm.pick[2]) {
    const uint32_t n = sm.pick[2];
    const bool listed = n <= kFewKeys;  // on the first CTA, which looks through the list alone
    if (listed) {
      // each CTA's own first; then to their place behind the first CTA's (one after the other, from every thread that
      // has one, they took 8000 clocks)
      if (rank != 0 && tid == 0) sm.cta_n[0] = 0;
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kPer; ++k)
        if (key[k] >> (32 - kTopBits) == limit >> (32 - kTopBits)) few[atomicAdd(&sm.cta_n[0], 1u)] = key[k];
      if (nranks > 1) {
        cluster_sync();
        if (rank != 0) {
          uint32_t to = 0;
          for (uint32_t c = 0; c < rank; ++c) to += ld_cluster_u32(mapa_shared(smem_u32(&sm.cta_n[0]), c));
          for (uint32_t i = tid; i < sm.cta_n[0]; i += kSelThreads)
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_shared(smem_u32(few + to + i), 0)), "r"(few[i]) : "memory");
        }
        cluster_sync();
      }
    }
    if (!listed || rank == 0) {
#pragma unroll 1
      for (int d = 0; d < 3; ++d) {  // 8, 8 and 4 bits
        const int shift = d == 0 ? 12 : d == 1 ? 4 : 0, above = shift + (d == 2 ? 4 : 8);
        const uint32_t bins = (1u << (above - shift)) - 1;
        clear_hist(sm);
        if (listed) {
          for (uint32_t i = tid; i < n; i += kSelThreads) {
            const uint32_t x = few[i];
            if ((x ^ limit) >> above == 0) count_digit(sm, x >> shift & bins);
          }
        } else {
#pragma unroll
          for (int k = 0; k < kPer; ++k)
            if ((key[k] ^ limit) >> above == 0) count_digit(sm, key[k] >> shift & bins);
        }
        choose_bin(sm, d, want, listed ? 1 : nranks);
        limit |= sm.pick[0] << shift;
        want = sm.pick[1];
        if (want == sm.pick[2]) break;
        if (listed && d == 0 && sm.pick[2] <= 32) {  // as few as that are ranked one against another
          const uint32_t last = sm.pick[2];
          if (tid == 0) sm.cta_n[1] = 0;
          __syncthreads();
          for (uint32_t i = tid; i < n; i += kSelThreads) {
            const uint32_t x = few[i];
            if ((x ^ limit) >> shift == 0) sm.all[atomicAdd(&sm.cta_n[1], 1u)] = x;
          }
          __syncthreads();
          if (warp == 0) {
            const uint32_t mine = lane < last ? sm.all[lane] : 0u;
            uint32_t gt = 0, ge = 0;
            for (uint32_t i = 0; i < last; ++i) {
              const uint32_t other = __shfl_sync(0xffffffffu, mine, i);
              gt += other > mine;
              ge += other >= mine;
            }
            if (lane < last && gt < want && want <= ge) {  // the want-th largest and its equals: the same answer
              sm.pick[0] = mine;
              sm.pick[1] = want - gt;
              sm.pick[2] = ge - gt;
            }
          }
          __syncthreads();
          limit = sm.pick[0];
          want = sm.pick[1];
          break;
        }
      }
    }
    if (listed && nranks > 1) {  // the first CTA's answer
      if (rank == 0 && tid == 0) sm.all[0] = limit;
      cluster_sync();
      limit = ld_cluster_u32(mapa_shared(smem_u32(&sm.all[0]), 0));
      want = ld_cluster_u32(mapa_shared(smem_u32(&sm.pick[1]), 0));
      const uint32_t in_bin = ld_cluster_u32(mapa_shared(smem_u32(&sm.pick[2]), 0));
      if (rank != 0) {
        __syncthreads();  // all have read their own
        if (tid == 0) sm.pick[2] = in_bin;
        __syncthreads();
      }
    }
  }
  if (want == sm.pick[2]) {  // the whole bin stays: every key from `limit` on
    limit = limit ? limit - 1 : 0;
    want = 0;
  }
  // keys above the limit stay, and the first `want` of those at it
  uint32_t gt = 0, eq = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) gt += __popc(__ballot_sync(0xffffffffu, key[k] > limit));
  if (want)
#pragma unroll
    for (int k = 0; k < kPer; ++k) eq += __popc(__ballot_sync(0xffffffffu, key[k] == limit));
  __syncthreads();  // warp_s has been read
  if (lane == 0) warp_s[warp] = gt | eq << 16;
  __syncthreads();
  uint32_t before = 0, total = 0;
  for (int i = 0; i < kSelWarps; ++i) {
    const uint32_t c = warp_s[i];
    if (i < warp) before += c;
    total += c;
  }
  gt = before & 0xFFFFu;
  eq = before >> 16;
  if (nranks > 1) {
    if (tid == 0) {
      sm.cta_n[0] = total & 0xFFFFu;
      sm.cta_n[1] = total >> 16;
    }
    cluster_sync();
    for (uint32_t c = 0; c < rank; ++c) {
      gt += ld_cluster_u32(mapa_shared(smem_u32(&sm.cta_n[0]), c));
      eq += ld_cluster_u32(mapa_shared(smem_u32(&sm.cta_n[1]), c));
    }
  }
  int32_t* kept = a.kept + unit * a.kept_stride + u.ns;
  const uint32_t below = (1u << lane) - 1;
  const int32_t row = u.lo + i0;
  if (want == 0) {  // no tie to cut
    kept += gt;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const uint32_t bg = __ballot_sync(0xffffffffu, key[k] > limit);
      if (key[k] > limit) kept[__popc(bg & below)] = row + 32 * k;
      kept += __popc(bg);
    }
  } else {
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const uint32_t bg = __ballot_sync(0xffffffffu, key[k] > limit), be = __ballot_sync(0xffffffffu, key[k] == limit);
      const uint32_t e = eq + __popc(be & below);
      if (key[k] > limit || (key[k] == limit && e < want)) kept[gt + __popc(bg & below) + min(e, want)] = row + 32 * k;
      gt += __popc(bg);
      eq += __popc(be);
    }
  }
  if (nranks > 1) cluster_sync();  // no CTA leaves while its counts are read
}

// Longer units: the weights are read six times, mostly from L2.
__global__ void __launch_bounds__(kSelThreads) select_long_kernel(SelectArgs a) {
  __shared__ __align__(16) SelectSmem sm;
  __shared__ uint32_t warp_gt[kSelWarps], warp_eq[kSelWarps];
  const uint32_t rank = cluster_ctarank(), nranks = cluster_nctarank();
  const int64_t unit = blockIdx.x / nranks;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Unit u;
  if (!select_begin(a, unit, rank, nranks, &u)) return;
  const int64_t len = u.hi - u.lo, per = ((len + nranks - 1) / nranks + 31) / 32 * 32;
  const int32_t c0 = (int32_t)(rank * per < len ? rank * per : len), c1 = (int32_t)(c0 + per < len ? c0 + per : len);
  const float* w = a.weights + unit * a.w_stride + u.lo;
  uint32_t limit = 0, want = u.want;
#pragma unroll 1
  for (int d = 0; d < kDigits; ++d) {
    const int shift = 24 - 8 * d;
    const uint32_t mask = d ? 0xFFFFFFFFu << (shift + 8) : 0u;
    clear_hist(sm);
#pragma unroll 8
    for (int32_t i = c0 + tid; i < c1; i += kSelThreads) {
      const uint32_t k = order_key(w[i]);
      if ((k & mask) == limit) count_digit(sm, (k >> shift) & 255u);
    }
    choose_bin(sm, d, want, nranks);
    limit |= sm.pick[0] << shift;
    want = sm.pick[1];
  }
  const int32_t perw = ((c1 - c0 + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
  const int32_t w0 = min(c0 + warp * perw, c1), w1 = min(w0 + perw, c1);
  int gt = 0, eq = 0;
#pragma unroll 8
  for (int32_t i = w0 + lane; i < w1; i += 32) {
    const uint32_t k = order_key(w[i]);
    gt += k > limit;
    eq += k == limit;
  }
  gt = warp_sum(gt);
  eq = warp_sum(eq);
  if (lane == 0) {
    warp_gt[warp] = gt;
    warp_eq[warp] = eq;
  }
  __syncthreads();
  if (tid == 0) {
    uint32_t sg = 0, se = 0;
    for (int i = 0; i < kSelWarps; ++i) {
      sg += warp_gt[i];
      se += warp_eq[i];
    }
    sm.cta_n[0] = sg;
    sm.cta_n[1] = se;
  }
  uint32_t gt0 = 0, eq0 = 0;  // rows above and at the limit before this warp's
  if (nranks > 1) {
    cluster_sync();
    for (uint32_t c = 0; c < rank; ++c) {
      gt0 += ld_cluster_u32(mapa_shared(smem_u32(&sm.cta_n[0]), c));
      eq0 += ld_cluster_u32(mapa_shared(smem_u32(&sm.cta_n[1]), c));
    }
  }
  for (int i = 0; i < warp; ++i) {
    gt0 += warp_gt[i];
    eq0 += warp_eq[i];
  }
  int32_t* kept = a.kept + unit * a.kept_stride + u.ns;
  const uint32_t below = (1u << lane) - 1;
#pragma unroll 4
  for (int32_t i = w0; i < w1; i += 32) {
    const bool in = i + lane < w1;
    const uint32_t k = in ? order_key(w[i + lane]) : 0u;
    const uint32_t bg = __ballot_sync(0xffffffffu, in && k > limit), be = __ballot_sync(0xffffffffu, in && k == limit);
    const uint32_t at_eq = eq0 + __popc(be & below);
    if (in && (k > limit || (k == limit && at_eq < want)))
      kept[gt0 + __popc(bg & below) + min(at_eq, want)] = u.lo + i + lane;
    gt0 += __popc(bg);
    eq0 += __popc(be);
  }
  if (nranks > 1) cluster_sync();  // no CTA leaves while its counts are read
}

// ---------------------------------------------------------------- mark
constexpr int kMarkThreads = 256;

__global__ void __launch_bounds__(kMarkThreads) mark_kernel(Layout L, int32_t shard_begin, int32_t B,
                                                            const int64_t* __restrict__ from_lens,
                                                            const int64_t* __restrict__ seq_lens, float* weights,
                                                            int64_t w_stride) {
  const int64_t unit = blockIdx.x;
  const int rs = (int)(unit / B), b = (int)(unit % B);
  const int64_t F = from_lens[b], S = seq_lens[b], r = shard_begin + rs;
  const int64_t first = F > 0 ? rows_below(r, F, L) : 0, n = S > 0 ? min(rows_below(r, S, L), w_stride) : 0;
  float* w = weights + unit * w_stride;
  for (int64_t i = first + blockIdx.y * kMarkThreads + threadIdx.x; i < n; i += gridDim.y * kMarkThreads) w[i] = INFINITY;
}

// ---------------------------------------------------------------- compact
struct CompactArgs {
  Layout L;
  int32_t shard_begin, n_held, B;
  const int32_t* kept;
  int64_t kept_stride;
  const int64_t* new_lens;
  const int32_t* bt;
  int64_t bt_stride, max_pages;
  unsigned char* arena;
  int64_t pool_pages;
  float* weights;  // may be null
  int64_t w_stride;
  int32_t* status;
};

// kWarps warps a CTA, each with a ring of kWindows windows of kRows rows (a lane each).
template <int kRowBytes, int kWarps_, int kRows_, int kWindows_>
struct Ring {
  static constexpr int kBytes = kRowBytes, kWarps = kWarps_, kRows = kRows_, kWindows = kWindows_;
  static constexpr int kSlotBytes = kRows * kRowBytes, kRingBytes = kWindows * kSlotBytes;
  static constexpr int kSmem = kWarps * kRingBytes;
  static_assert(kRows <= 32 && kWindows >= 4, "a lane a row; two windows in flight beside the two being stored");
};

__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(reinterpret_cast<uint64_t>(dst)),
               "r"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kPending) : "memory");
}
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// 4 bytes of global memory into shared memory, and an arrival on `bar` when this
// thread's copies so far have landed.
__device__ __forceinline__ void copy4_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)) : "memory");
}
__device__ __forceinline__ void copies_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

template <class R>
__global__ void __launch_bounds__(32 * R::kWarps) compact_kernel(CompactArgs a) {
  constexpr int kRowBytes = R::kBytes;
  extern __shared__ __align__(128) unsigned char rings[];
  __shared__ uint64_t fulls[R::kWarps][R::kWindows];
  __shared__ float w_all[R::kWarps][R::kWindows][R::kRows];
  __shared__ int abort_w;
  volatile int* abort_s = &abort_w;
  uint32_t nranks = cluster_nctarank();
  const int64_t u = blockIdx.x / nranks;
  const int rs = (int)(u / a.B), b = (int)(u % a.B), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t M = a.new_lens[b];
  const int64_t m64 = M > 0 ? rows_below(a.shard_begin + rs, M, a.L) : 0;
  if (M < 0 || m64 > a.kept_stride) {  // uniform over the cluster
    if (threadIdx.x == 0 && cluster_ctarank() == 0) flag(a.status, DCP_STATUS_BAD_LENGTH);
    return;
  }
  const int32_t m = (int32_t)m64;
  if (m == 0) return;
  // a window of the unit is one of every warp of the cluster
  const uint32_t rank = cluster_ctarank() * R::kWarps + warp;
  nranks *= R::kWarps;
  unsigned char* ring = rings + warp * R::kRingBytes;
  uint64_t* full = fulls[warp];
  float (*w_s)[R::kRows] = w_all[warp];
  if (threadIdx.x == 0) *abort_s = 0;
  if (lane == 0) {
    for (int i = 0; i < R::kWindows; ++i) mbar_init(&full[i], 33);  // the byte count, and every lane's weight
    fence_barrier_init();
  }
  __syncthreads();
  const int32_t* kept = a.kept + u * a.kept_stride;
  const int32_t* bt = a.bt + (int64_t)b * a.bt_stride;
  float* wts = a.weights ? a.weights + u * a.w_stride : nullptr;
  unsigned char* pool = a.arena + rs * a.pool_pages * a.L.P * kRowBytes;
  const int32_t P = (int32_t)a.L.P;
  const int32_t shift = (P & (P - 1)) ? -1 : 31 - __clz(P);  // page sizes are mostly powers of two
  auto page_at = [&](int32_t row) -> int32_t { return shift >= 0 ? row >> shift : row / P; };
  auto in_page = [&](int32_t row) -> int32_t { return shift >= 0 ? row & (P - 1) : row % P; };
  const int32_t step = (int32_t)nranks * R::kRows;
  const int32_t nwin = (int32_t)(((int64_t)m + step - 1) / step);

  // Window x's row of this lane: i = x * step + rank * kRows + lane.  Its kept entry is
  // loaded two windows ahead of its copy and its two pages one ahead.
  auto row_at = [&](int32_t x) -> int64_t { return (int64_t)x * step + rank * R::kRows + lane; };
  auto load_kept = [&](int32_t x) -> int32_t {
    const int64_t i = row_at(x);
    return lane < R::kRows && i < m ? __ldg(kept + i) : -1;
  };
  struct Pages {
    int32_t from, src, dst;  // row moved from (-1: none), its page and that of its place
  };
  auto load_pages = [&](int32_t x, int32_t k) -> Pages {
    const int64_t i = row_at(x);
    if (k < 0 || k <= i) {
      if (k < -1 || (k >= 0 && k < i)) flag(a.status, DCP_STATUS_BAD_POSITION);
      return Pages{-1, 0, 0};  // none, or in its place already
    }
    if (page_at(k) >= a.max_pages || (wts && k >= a.w_stride)) {
      flag(a.status, DCP_STATUS_BAD_PAGE_INDEX);
      return Pages{-1, 0, 0};
    }
    return Pages{k, __ldg(bt + page_at(k)), __ldg(bt + page_at((int32_t)i))};
  };
  // window x into its slot; returns where this lane's row goes (null: nowhere)
  auto load = [&](int32_t x, const Pages& pg) -> unsigned char* {
    const int s = x % R::kWindows;
    const int32_t i = (int32_t)row_at(x);
    bool live = pg.from >= 0;
    if (live && (pg.src < 0 || pg.src >= a.pool_pages || pg.dst < 0 || pg.dst >= a.pool_pages)) {
      flag(a.status, DCP_STATUS_BAD_PAGE_ID);
      live = false;
    }
    const uint32_t who = __ballot_sync(0xffffffffu, live);
    if (lane == 0) mbar_arrive_expect_tx(&full[s], __popc(who) * kRowBytes);
    __syncwarp();
    if (live) {
      bulk_load(ring + s * R::kSlotBytes + lane * kRowBytes, pool + ((int64_t)pg.src * P + in_page(pg.from)) * kRowBytes,
                kRowBytes, &full[s]);
      if (wts) copy4_async(smem_u32(&w_s[s][lane]), wts + pg.from);
    }
    copies_arrive(&full[s]);
    return live ? pool + ((int64_t)pg.dst * P + in_page(i)) * kRowBytes : nullptr;
  };

  constexpr int kAhead = R::kWindows - 2;  // windows loaded ahead of the one written
  unsigned char* dst[R::kWindows];
  int32_t k1 = load_kept(0), k2 = load_kept(1);
  Pages pg = load_pages(0, k1);
  k1 = k2;
  k2 = load_kept(2);
  // windows in groups of kWindows, so that `dst` stays in registers
  auto feed = [&](int32_t x) -> unsigned char* {  // window x, whose pages are in flight; fetches ahead
    unsigned char* to = load(x, pg);
    pg = load_pages(x + 1, k1);
    k1 = k2;
    k2 = load_kept(x + 3);
    return to;
  };
#pragma unroll
  for (int x = 0; x < kAhead; ++x) dst[x] = x < nwin ? feed(x) : nullptr;
  // The barrier that says "window x has been read by all" is arrived at a window early, so that it completes behind
  // the store and the copies of the window before.  It orders no memory: the rows have landed when a CTA arrives.
  bool ok = true;
  auto read_one = [&](int s, int32_t x) {
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&full[s], (uint32_t)(x / R::kWindows) & 1u, abort_s));
    __syncwarp();
    if (nranks > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // after a lost wait too
  };
  read_one(0, 0);
  for (int32_t x0 = 0; x0 < nwin; x0 += R::kWindows) {
#pragma unroll
    for (int s = 0; s < R::kWindows; ++s) {
      const int32_t x = x0 + s;
      if (x >= nwin) break;
      const bool had = ok;
      if (nranks > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
      if (x + 1 < nwin) read_one((s + 1) % R::kWindows, x + 1);
      if (had) {
        if (dst[s]) {
          bulk_store(dst[s], smem_u32(ring) + s * R::kSlotBytes + lane * kRowBytes, kRowBytes);
          if (wts) wts[row_at(x)] = w_s[s][lane];
        }
        bulk_commit();
      }
      if (ok && x + kAhead < nwin) {
        bulk_wait_read<2>();  // window x - 2 has left the slot that is filled next
        dst[(s + kAhead) % R::kWindows] = feed(x + kAhead);
      }
    }
  }
  bulk_wait_all();
  if (!ok) {
    if (lane == 0) flag(a.status, DCP_STATUS_TIMEOUT);
    const uint64_t t0 = globaltimer();  // copies in flight land before the block's memory is given back
    while (globaltimer() - t0 < 100000) {
    }
  }
}

bool shards_ok(const dcp_layout_t* layout, int32_t shard_begin, int32_t shard_end, int32_t B) {
  return layout_ok(layout) && shard_begin >= 0 && shard_end <= layout->n_shards && shard_begin < shard_end && B >= 1;
}

// CTAs a unit: doubled while the units alone leave SMs idle and every CTA keeps `least` rows.
unsigned cluster_of(int64_t units, int64_t rows, int64_t least, int64_t fill) {
  unsigned c = 1;
  while (c < 8 && units * c * 2 <= fill && rows / (c * 2) >= least) c *= 2;
  return c;
}

template <class Kernel, class Args>
int32_t launch_clusters(Kernel kernel, int64_t units, unsigned c, int threads, size_t smem, void* stream, const Args& a) {
  if (units * c > INT32_MAX) return DCP_ERR_UNSUPPORTED;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = c;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)(units * c));
  lc.blockDim = dim3(threads);
  lc.dynamicSmemBytes = smem;
  lc.stream = as_stream(stream);
  lc.attrs = at;
  lc.numAttrs = 1;
  if (cudaLaunchKernelEx(&lc, kernel, a) != cudaSuccess) return DCP_ERR_CUDA;
  return launch_status();
}

template <class R>
int32_t launch_compact(int64_t units, unsigned c, void* stream, const CompactArgs& a) {
  static SmemLimit limit;
  if (!limit.ensure(reinterpret_cast<const void*>(&compact_kernel<R>), R::kSmem)) return DCP_ERR_CUDA;
  return launch_clusters(compact_kernel<R>, units, c, 32 * R::kWarps, R::kSmem, stream, a);
}

// A bulk copy's operands are uniform ones: a warp issues its lanes' copies one after the other, some 75 ns each, so
// eight warps an SM are wanted.  One warp a CTA, eight CTAs an SM, where the units are enough for that with up to 8 CTAs
// each; else eight warps a CTA.  524288 rows kept, in us, 8 CTAs an SM / 8 warps a CTA: 128 units 195 / 204 (4-bit 236 /
// 242), 64 units 292 / 205; 262144 rows of 16 units 539 / 184 (385 / 172).  Four warps an SM, in windows of twice the
// rows: 203 (249); one warp an SM in windows of 32 rows: 305 (471).
template <class Many, class Few>
int32_t compact(const dcp_layout_t* layout, int32_t shard_begin, int32_t shard_end, const int32_t* kept,
                int64_t kept_stride, int32_t B, const int64_t* new_lens, const int32_t* block_table,
                int64_t bt_stride, int64_t max_pages, void* arena, int64_t pool_pages, float* weights,
                int64_t w_stride, int32_t* status, void* stream) {
  if (!shards_ok(layout, shard_begin, shard_end, B) || kept_stride < 0 || max_pages < 1 || bt_stride < max_pages ||
      pool_pages < 1 || (weights && w_stride < 1))
    return DCP_ERR_INVALID;
  if (!new_lens || !block_table || !arena || (kept_stride && !kept) || (reinterpret_cast<uintptr_t>(arena) & 15))
    return DCP_ERR_INVALID;
  if (kept_stride == 0) return DCP_OK;
  if (kept_stride > INT32_MAX - 1024) return DCP_ERR_UNSUPPORTED;  // kept entries are 32-bit rows
  const CompactArgs a{to_layout(layout), shard_begin, shard_end - shard_begin, B, kept, kept_stride, new_lens,
                      block_table, bt_stride, max_pages, static_cast<unsigned char*>(arena), pool_pages, weights,
                      w_stride, status};
  const int64_t units = (int64_t)B * a.n_held;
  if (units * 8 >= 1024)
    return launch_compact<Many>(units, cluster_of(units, kept_stride, 2 * Many::kRows, 1216), stream, a);
  return launch_compact<Few>(units, cluster_of(units, kept_stride, 2 * Few::kRows * Few::kWarps, 152), stream, a);
}

}  // namespace

extern "C" int32_t dcp_key_weights_mark(const dcp_layout_t* layout, int32_t shard_begin, int32_t shard_end, int32_t B,
                                        const int64_t* from_lens, const int64_t* seq_lens, float* weights,
                                        int64_t w_stride, void* stream) {
  if (!shards_ok(layout, shard_begin, shard_end, B) || w_stride < 1) return DCP_ERR_INVALID;
  if (!from_lens || !seq_lens || !weights) return DCP_ERR_INVALID;
  const int64_t units = (int64_t)B * (shard_end - shard_begin);
  if (units > INT32_MAX) return DCP_ERR_UNSUPPORTED;
  // A call marks a few rows as a rule, one trip of one block: more blocks a unit (for a cache that was never weighed) only
  // while the units leave SMs idle.
  const unsigned parts = (unsigned)std::min<int64_t>((w_stride + 16 * kMarkThreads - 1) / (16 * kMarkThreads),
                                                     std::max<int64_t>(1, 304 / units));
  mark_kernel<<<dim3((unsigned)units, parts), kMarkThreads, 0, as_stream(stream)>>>(
      to_layout(layout), shard_begin, B, from_lens, seq_lens, weights, w_stride);
  return launch_status();
}

extern "C" int32_t dcp_evict_select(const dcp_layout_t* layout, int32_t shard_begin, int32_t shard_end, int32_t B,
                                    const int64_t* seq_lens, const int64_t* new_lens, int64_t sinks, int64_t recent,
                                    const float* weights, int64_t w_stride, int32_t* kept, int64_t kept_stride,
                                    int32_t* status, void* stream) {
  if (!shards_ok(layout, shard_begin, shard_end, B) || sinks < 0 || recent < 0 || w_stride < 1 || kept_stride < 1)
    return DCP_ERR_INVALID;
  if (!seq_lens || !new_lens || !weights || !kept) return DCP_ERR_INVALID;
  if (w_stride > INT32_MAX - 1024) return DCP_ERR_UNSUPPORTED;
  const SelectArgs a{to_layout(layout), shard_begin, shard_end - shard_begin, B, seq_lens, new_lens, sinks, recent,
                     weights, w_stride, kept, kept_stride, status};
  const int64_t units = (int64_t)B * a.n_held;
  // CTAs a unit while they leave SMs idle, then as many as hold its rows in registers
  unsigned c = cluster_of(units, w_stride, 2048, 304);
  while (c < 8 && w_stride > (int64_t)c * 32 * kSelThreads) c *= 2;
  const int64_t per = (w_stride + c * kSelThreads - 1) / (c * kSelThreads);
  const auto kernel = per <= 4 ? select_kernel<4> : per <= 16 ? select_kernel<16> : per <= 32 ? select_kernel<32> : select_long_kernel;
  return launch_clusters(kernel, units, c, kSelThreads, 0, stream, a);
}

extern "C" int32_t dcp_kv_compact(const dcp_layout_t* layout, int32_t shard_begin, int32_t shard_end,
                                  const int32_t* kept, int64_t kept_stride, int32_t B, const int64_t* new_lens,
                                  const int32_t* block_table, int64_t bt_stride, int64_t max_pages, void* arena,
                                  int64_t pool_pages, float* weights, int64_t w_stride, int32_t* status,
                                  void* stream) {
  return compact<Ring<kDk * 2, 1, 4, 6>, Ring<kDk * 2, 8, 4, 6>>(layout, shard_begin, shard_end, kept, kept_stride, B, new_lens, block_table,
                          bt_stride, max_pages, arena, pool_pages, weights, w_stride, status, stream);
}

extern "C" int32_t dcp_kv_compact_q4(const dcp_layout_t* layout, int32_t shard_begin, int32_t shard_end,
                                     const int32_t* kept, int64_t kept_stride, int32_t B, const int64_t* new_lens,
                                     const int32_t* block_table, int64_t bt_stride, int64_t max_pages, void* arena,
                                     int64_t pool_pages, float* weights, int64_t w_stride, int32_t* status,
                                     void* stream) {
  return compact<Ring<kQ4RowBytes, 1, 8, 8>, Ring<kQ4RowBytes, 8, 8, 8>>(layout, shard_begin, shard_end, kept, kept_stride, B, new_lens, block_table,
                              bt_stride, max_pages, arena, pool_pages, weights, w_stride, status, stream);
}
