// dcp_decode.cuh — what the partial-attention kernels share: the stream-K work
// split and its planner, the softmax helpers, the output rows, the merge of cut
// units and the host-side checks and launches.  dcp_decode.cu attends over a bf16
// cache, dcp_decode_q4.cu over a 4-bit one; each holds its own main kernel.
//
// Work split (stream-K): units are (request, shard); unit u has T_u tiles.  The
// concatenation of all units' tiles is cut into V equal ranges, one per cluster
// (per row group).  A unit inside one range is written directly; a unit cut by
// range boundaries leaves normalised pieces (o, lse in base 2) in the workspace
// which a second kernel merges with the same LSE rule.  A tiny kernel run first
// writes the tile prefix sums.
#pragma once

#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "dcp_internal.cuh"
#include "sm100_ptx.cuh"

using namespace dcp;
using namespace dcp::sm100;

namespace {

constexpr int kTile = 64;                     // KV rows per tile
constexpr int kChunkDims = 64;                // dims per chunk (one 128-byte swizzle row)
constexpr int kChunkBytes = kTile * 128;      // 8 KB
constexpr int kOwnChunks = 4;                 // value chunks each CTA of a pair holds (256 dims)
constexpr int kRopeHalf = 32;                 // rope dims each CTA holds (64-byte swizzled rows)
constexpr int kRopeHalfBytes = kTile * 64;
constexpr int kRopeOff = kOwnChunks * kChunkBytes;         // rope part inside a tile slot
constexpr int kSlotBytes = kRopeOff + kRopeHalfBytes;      // 36 KB per tile slot
constexpr int kHalfRows = 16;                 // rows served by one softmax warp (two threads per row)
constexpr int kMaxGroupRows = 128;
constexpr int64_t kMaxQueryRows = 65536;      // q_len * H per request (512 row groups)
constexpr int64_t kMaxUnitRows = 1 << 30;     // rows of a unit; a pool of more is beyond any card's memory
constexpr int kXRowBytes = kTile * 4;         // one row of a partial score tile (fp32)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.0f;     // log2 units: P stays <= 256
constexpr size_t kSmemBudget = 232448;        // 227 KB

struct TcArgs {
  Layout L;
  int32_t shard_begin, n_held;
  int32_t B, q_len, H, R_total;  // R_total = q_len * H
  int32_t Rg, ngroups, V;        // rows per group, groups, stream-K ranges
  int32_t nts;                   // tile slots in the ring
  int32_t nraw;                  // raw tiles of a 4-bit cache in flight
  int32_t box_rows;              // KV TMA box height = min(P, 64)
  int64_t pool_rows, pool_pages;
  int64_t max_rows;              // rows a unit's table row can hold: no more are looked at, whatever its length says
  const int32_t* bt;
  int64_t bt_stride, max_pages;
  const int64_t* seq_lens;
  float scale_log2;
  int32_t base2;
  void* o_part;
  int32_t o_bf16;
  float* lse_part;
  const __nv_bfloat16* q;     // [B * R_total][576]
  const int32_t* tile_start;  // [U + 1]
  float* piece_o;             // [2V][R_total][512]
  float* piece_lse;           // [2V][R_total]
  int32_t* status;
};
__host__ __device__ inline uint32_t round1024(uint32_t v) { return (v + 1023u) & ~1023u; }

__device__ inline int64_t unit_nvis_max(const TcArgs& a, int b, int rs, bool* bad) {
  const int64_t S = a.seq_lens[b];
  if (S < a.q_len) {
    *bad = true;
    return 0;
  }
  return count_of(a.shard_begin + rs, S, a.L);
}

// ---------------------------------------------------------------------------- planner
// Tile prefix sums of the (request, shard) units, and the rows of units with no
// visible key (an empty shard): o = 0 and lse = -inf, written here because the
// main kernel never visits them.  One block of 1024 threads, 1024 units per pass.
__global__ void __launch_bounds__(1024) plan_kernel(TcArgs a, int32_t* tile_start, int32_t U) {
  __shared__ int32_t warp_sums[32];
  __shared__ int32_t carry;
  __shared__ int32_t empty_s[1024];
  __shared__ int32_t n_empty_s;
  if (threadIdx.x == 0) {
    carry = 0;
    n_empty_s = 0;
  }
  __syncthreads();
  for (int32_t base = 0; base < U; base += 1024) {
    const int32_t u = base + threadIdx.x;
    int32_t t = 0;
    if (u < U) {
      bool bad = false;
      const int b = u / a.n_held, rs = u % a.n_held;
      int64_t n = unit_nvis_max(a, b, rs, &bad);
      if (bad && rs == 0) flag(a.status, DCP_STATUS_BAD_LENGTH);
      if (n > a.max_rows) {
        flag(a.status, DCP_STATUS_BAD_PAGE_ID);  // pages past the table
        n = a.max_rows;
      }
      t = (int32_t)((n + kTile - 1) / kTile);
      if (t == 0) empty_s[atomicAdd(&n_empty_s, 1)] = u;  // at most 1024 per pass
    }
    // block-wide inclusive scan
    int32_t x = t;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      int32_t y = __shfl_up_sync(0xffffffffu, x, s);
      if (lane >= s) x += y;
    }
    if (lane == 31) warp_sums[w] = x;
    __syncthreads();
    if (w == 0) {
      int32_t ws = warp_sums[lane];
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        int32_t y = __shfl_up_sync(0xffffffffu, ws, s);
        if (lane >= s) ws += y;
      }
      warp_sums[lane] = ws;
    }
    __syncthreads();
    const int32_t incl = x + (w > 0 ? warp_sums[w - 1] : 0) + carry;
    if (u < U) tile_start[u] = incl - t;
    __syncthreads();
    if (threadIdx.x == 1023) carry = incl;
    // this pass's empty units: every thread writes 16-byte pieces of their rows
    const int n_empty = n_empty_s;
    const int64_t row_bytes = (int64_t)kDv * (a.o_bf16 ? 2 : 4);
    for (int k = 0; k < n_empty; ++k) {
      const int32_t ue = empty_s[k];
      const int64_t row0 = ((int64_t)(ue % a.n_held) * a.B + ue / a.n_held) * a.R_total;
      uint4* dst = reinterpret_cast<uint4*>(static_cast<unsigned char*>(a.o_part) + row0 * row_bytes);
      for (int64_t i = threadIdx.x; i < a.R_total * row_bytes / 16; i += 1024) dst[i] = make_uint4(0, 0, 0, 0);
      for (int i = threadIdx.x; i < a.R_total; i += 1024) a.lse_part[row0 + i] = -INFINITY;
    }
    __syncthreads();
    if (threadIdx.x == 0) n_empty_s = 0;
    __syncthreads();
  }
  if (threadIdx.x == 0) tile_start[U] = carry;
}

// ---------------------------------------------------------------------------- segments
// A CTA's range [lo, hi) of the global tile sequence, visited unit by unit.
struct SegIter {
  const int32_t* start;
  int32_t U;
  int64_t lo, hi;
  int32_t u;

  __device__ void init(const int32_t* st, int32_t nunits, int64_t lo_, int64_t hi_) {
    start = st; U = nunits; lo = lo_; hi = hi_;
    // largest u with start[u] <= lo
    int32_t l = 0, h = U;  // start[U] = total > lo when lo < hi
    while (h - l > 1) {
      const int32_t m = (l + h) >> 1;
      if (start[m] <= lo) l = m; else h = m;
    }
    u = l;
  }
  // next segment: unit, first tile (within the unit), tile count, whole-unit flag, piece slot
  __device__ bool next(int32_t* unit, int32_t* t0, int32_t* nt, bool* whole, int* kslot) {
    while (u < U) {
      const int64_t s = start[u], e = start[u + 1];
      if (s >= hi) return false;
      const int64_t a = s > lo ? s : lo, b = e < hi ? e : hi;
      const int32_t cur = u++;
      if (a < b) {
        *unit = cur;
        *t0 = (int32_t)(a - s);
        *nt = (int32_t)(b - a);
        *whole = (a == s) && (b == e);
        *kslot = (a == lo) ? 0 : 1;
        return true;
      }
    }
    return false;
  }
};

// First tile of range v of V (32-bit division where it does: a 64-bit one is some
// hundred instructions, and the fixup makes a chain of them).
__device__ __forceinline__ int64_t div_tiles(int64_t x, int64_t by) {
  return ((x | by) >> 31) == 0 ? (int64_t)((uint32_t)x / (uint32_t)by) : x / by;
}
__device__ inline int64_t range_lo(int64_t T, int v, int V) { return div_tiles(T * v, V); }

// Two fp32 values in one 64-bit register pair, for the packed FP32 operations
// of sm_100 (two lanes per instruction; each lane rounds as its scalar form).
__device__ __forceinline__ uint64_t f2_pack(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ void f2_unpack(uint64_t v, uint32_t& lo, uint32_t& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// The largest of three values, or NaN if one of them is.
__device__ __forceinline__ float fmax3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// 2^x with the hardware approximation (ex2.approx.ftz: relative error ~2^-22,
// 2^-inf = +0); the result is rounded to bf16 for the PV product anyway.
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Warp-uniform bounded waits.  Fast path: every lane tests the phase once (its
// own acquire) and one vote confirms; otherwise each lane waits with the bounded
// loop and a final vote makes the outcome uniform (false after an abort).
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_s, int lane) {
  bool ok = mbar_try_wait(bar, parity);  // every lane: its own acquire
  if (__all_sync(0xffffffffu, ok)) return true;
  if (!ok) ok = mbar_wait(bar, parity, abort_s);
  return __all_sync(0xffffffffu, ok);  // warp-uniform (false after an abort)
}

__device__ __forceinline__ bool warp_wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort_s, int lane) {
  bool ok = mbar_try_wait_cluster(bar, parity);
  if (__all_sync(0xffffffffu, ok)) return true;
  if (!ok) ok = mbar_wait_cluster(bar, parity, abort_s);
  return __all_sync(0xffffffffu, ok);
}

// O rows of one softmax warp scaled by f (16 lanes from `o_addr`'s lane;
// thread t: row t % 16, columns [128 (t / 16), 128 (t / 16) + 128)).
__device__ __forceinline__ void rescale_rows(uint32_t o_addr, float f) {
#pragma unroll 1
  for (int k = 0; k < 4; ++k) {
    uint32_t r[32];
    tmem_ld16x2_sync<128>(o_addr + 32 * k, r);
#pragma unroll
    for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * f);
    tmem_st16x2<128>(o_addr + 32 * k, r);
    tmem_st_wait();  // before the next load reuses r
  }
}

// The same O rows times `inv` -> the output rows (bf16 or fp32) or the fp32
// piece rows; thread t holds dims [d0, d0 + 128) of row r0 + t % 16.  Rows
// [0, rows_here) of the group are written.  Kept out of line: it runs once per
// segment and inlining it cost the tile loop.
//
// fp32 rows go through `stage`, this warp's 16 rows of the score-exchange
// buffer it read the peer's last tile from (4 KB: 64 floats per row, 16-byte
// chunk c of row r at chunk slot c ^ (r % 16), as the exchange lays them out);
// nothing writes those rows again before this warp ships its next tile.  Per 32
// dims, each thread writes its row segment (128 bytes) there, and the warp reads
// them back so that 8 lanes hold one segment: each store instruction writes 4
// whole 128-byte lines.  (Each lane storing its own row touches 32 lines per
// instruction and took about twice as long; a shuffle transpose among lane
// groups of 4 touches 8 and spends more in shuffles than the staging costs.)
// bf16 rows go the same way, two 32-dim blocks (128 bytes) per thread at a
// time.  All global stores are 16 bytes wide: a 32-byte
// st.global.v8 in this routine was found to land only its first word in one
// build of the kernel.
__device__ __noinline__ void store_o_rows(const TcArgs& a, uint32_t o_addr, int rows_here, bool whole,
                                          int64_t out_base, int64_t piece_base, int r0, int d0, float inv,
                                          uint32_t stage) {
  const int lane = threadIdx.x & 31;
  const int h = lane >> 4, lr = lane & 15;          // this thread's half-row and row within the warp
  const int dbase = d0 - 128 * h;                   // this CTA's first dim
  const int c = lane & 7;                           // read-back: chunk c of segment 4 i + lane / 8
  if (whole && a.o_bf16) {
    // bf16 rows, staged like the fp32 ones: two 32-dim blocks (128 bytes) per
    // thread at a time
    __nv_bfloat16* const outb = static_cast<__nv_bfloat16*>(a.o_part) + out_base * kDv;
#pragma unroll 1
    for (int kp = 0; kp < 2; ++kp) {
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {        // each 32-dim block: 4 of the row segment's 8 chunks
        uint32_t rr[32];
        tmem_ld16x2_sync<128>(o_addr + 32 * (2 * kp + half), rr);
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          __nv_bfloat162 hh =
              __floats2bfloat162_rn(__uint_as_float(rr[2 * e]) * inv, __uint_as_float(rr[2 * e + 1]) * inv);
          w[e] = *reinterpret_cast<uint32_t*>(&hh);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          st_shared_v4(stage + (uint32_t)lr * kXRowBytes + ((uint32_t)((8 * h + 4 * half + i) ^ lr) << 4), w[4 * i],
                       w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int sg = 4 * i + (lane >> 3);         // segment: row sg / 2, half sg % 2
        const int sr = sg >> 1, sh = sg & 1;
        const uint4 v = ld_shared_v4(stage + (uint32_t)sr * kXRowBytes + ((uint32_t)((8 * sh + c) ^ sr) << 4));
        if (r0 + sr < rows_here)
          *reinterpret_cast<uint4*>(outb + (int64_t)(r0 + sr) * kDv + dbase + 128 * sh + 64 * kp + 8 * c) = v;
      }
      __syncwarp();
    }
    return;
  }
  float* const out0 = whole ? static_cast<float*>(a.o_part) + out_base * kDv : a.piece_o + piece_base * kDv;
#pragma unroll 1
  for (int k = 0; k < 4; ++k) {
    uint32_t rr[32];
    tmem_ld16x2_sync<128>(o_addr + 32 * k, rr);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      st_shared_v4(stage + (uint32_t)lr * kXRowBytes + ((uint32_t)((8 * h + i) ^ lr) << 4),
                   __float_as_uint(__uint_as_float(rr[4 * i]) * inv), __float_as_uint(__uint_as_float(rr[4 * i + 1]) * inv),
                   __float_as_uint(__uint_as_float(rr[4 * i + 2]) * inv), __float_as_uint(__uint_as_float(rr[4 * i + 3]) * inv));
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int sg = 4 * i + (lane >> 3);           // segment: row sg / 2, half sg % 2
      const int sr = sg >> 1, sh = sg & 1;
      const uint4 v = ld_shared_v4(stage + (uint32_t)sr * kXRowBytes + ((uint32_t)((8 * sh + c) ^ sr) << 4));
      if (r0 + sr < rows_here)
        *reinterpret_cast<uint4*>(out0 + (int64_t)(r0 + sr) * kDv + dbase + 128 * sh + 32 * k + 4 * c) = v;
    }
    __syncwarp();                                   // the reads are done before the next k's writes
  }
}

// Largest u in [0, U) with start[u] <= x, for a whole warp: 32 probes a step (a
// bisection is a chain of log2(U) loads: 2 us more for 256 units).
__device__ __forceinline__ int32_t find_unit(const int32_t* start, int32_t U, int64_t x) {
  const int lane = threadIdx.x & 31;
  int32_t l = 0, h = U;
  while (h - l > 1) {
    const int32_t step = (h - l + 31) / 32, m = l + step * lane;
    const uint32_t below = __ballot_sync(0xffffffffu, m < h && start[m] <= x);  // at least the first
    l += step * (31 - __clz(below));
    h = min(h, l + step);
  }
  return l;
}

// ---------------------------------------------------------------------------- fixup
// Merges the pieces of units cut by range boundaries (the same LSE rule as the
// shard merge, base 2).  Only range boundaries cut units, so block column k
// serves boundary k (between ranges k and k + 1): the unit containing that
// boundary's first tile, if the boundary falls inside it and no earlier boundary
// does (the first boundary inside a unit merges all its pieces).  Blocks per
// column: up to 12, each taking chunks of query rows; the first warp builds the
// unit's piece list in shared memory, then the warps merge the pieces with 16-byte
// loads and stores, a warp taking kQ quarters (128 dims) of a row and 8 / kQ pieces at
// a time.  Whole rows (kQ = 4) serve many rows of few pieces: with quarters the blocks
// are four times as many, 362 us against 348 for 32 requests of 32k tokens and 128
// heads.  Halves (kQ = 2) serve at most 16 rows, where one long request's unit has up to
// 38 pieces and a warp's loads are a chain.  Whole rows / halves / quarters, 8 heads:
// one request of 64k tokens 36 / 31 / 30 us, of 8k 21 / 18 / 18; 64 of 2k 45 / 44 / 48.
constexpr int kFixupThreads = 256;
constexpr int kMaxPieces = 512;

constexpr int kFixupWarps = kFixupThreads / 32;
constexpr int kFixupFewRows = 16;  // most rows that are merged by halves

template <int kQ>
__global__ void __launch_bounds__(kFixupThreads) fixup_kernel(TcArgs a) {
  constexpr int kAhead = 8 / kQ, kParts = kDv / 128 / kQ;
  __shared__ int32_t piece_s[kMaxPieces];
  __shared__ int32_t npiece_s, unit_s;
  griddep_wait();  // a programmatic dependent of the partial kernel: its pieces are complete after this
  const int32_t U = a.B * a.n_held;
  const int V = a.V;
  const int64_t T = a.tile_start[U];
  const int lane = threadIdx.x & 31;
  if (threadIdx.x < 32) {
    const int k = blockIdx.x;
    const int64_t x = range_lo(T, k + 1, V);  // the boundary's first tile
    int unit = -1;
    if (x > 0 && x < T) {
      const int32_t l = find_unit(a.tile_start, U, x);  // the unit u with start[u] <= x < start[u + 1]
      const int64_t su = a.tile_start[l];
      if (su < x && (k == 0 || range_lo(T, k, V) <= su)) unit = l;
    }
    if (lane == 0) unit_s = unit;
  }
  __syncthreads();
  const int32_t u = unit_s;
  if (u < 0) return;
  const int b = u / a.n_held, rs = u % a.n_held;
  const int64_t s = a.tile_start[u], e = a.tile_start[u + 1];
  const int64_t out_row0 = ((int64_t)rs * a.B + b) * a.R_total;
  if (threadIdx.x < 32) {
    auto part_of = [&](int64_t x) {  // range containing tile x
      int vv = (int)div_tiles(x * V, T);
      while (vv + 1 < V && range_lo(T, vv + 1, V) <= x) ++vv;
      while (vv > 0 && range_lo(T, vv, V) > x) --vv;
      return vv;
    };
    const int v0 = part_of(s), v1 = part_of(e - 1);
    int n = 0;
    if (v0 != v1) {
      for (int base = v0; base <= v1 && n < kMaxPieces; base += 32) {
        const int vv = base + lane;
        const int64_t rlo = range_lo(T, vv, V);
        const bool piece = vv <= v1 && rlo != range_lo(T, vv + 1, V);  // an empty range has none
        const uint32_t with = __ballot_sync(0xffffffffu, piece);
        const int at = n + __popc(with & ((1u << lane) - 1));
        if (piece && at < kMaxPieces) piece_s[at] = 2 * vv + (rlo >= s ? 0 : 1);
        n = min(n + __popc(with), kMaxPieces);
      }
    }
    if (lane == 0) npiece_s = n;
  }
  __syncthreads();
  const int np = npiece_s;
  const int items = a.R_total * kParts;
  for (int item = blockIdx.y * kFixupWarps + (threadIdx.x >> 5); item < items; item += gridDim.y * kFixupWarps) {
    const int row = item / kParts, d = item % kParts * (128 * kQ) + 4 * lane;  // and 128 on for each further quarter
    float m = -INFINITY;
    for (int k = lane; k < np; k += 32) m = fmax_nan(m, a.piece_lse[(int64_t)piece_s[k] * a.R_total + row]);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) m = fmax_nan(m, __shfl_xor_sync(0xffffffffu, m, x));
    float4 acc[kQ];
#pragma unroll
    for (int q = 0; q < kQ; ++q) acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
    float wsum = 0.f;
    if (m != -INFINITY) {
      for (int base = 0; base < np; base += kAhead) {
        float4 o[kAhead][kQ];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const float* src = a.piece_o + ((int64_t)piece_s[min(base + i, np - 1)] * a.R_total + row) * kDv + d;
#pragma unroll
          for (int q = 0; q < kQ; ++q)
            o[i][q] = base + i < np ? *reinterpret_cast<const float4*>(src + 128 * q) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        const float l = lane < kAhead && base + lane < np
                            ? a.piece_lse[(int64_t)piece_s[base + lane] * a.R_total + row]
                            : -INFINITY;
        const float w = l == -INFINITY ? 0.f : exp2f(l - m);  // lane i: piece base + i's
#pragma unroll
        for (int i = 0; i < kAhead; i += 2) {
          const float w0 = __shfl_sync(0xffffffffu, w, i), w1 = __shfl_sync(0xffffffffu, w, i + 1);
          wsum += w0 + w1;
#pragma unroll
          for (int q = 0; q < kQ; ++q) {
            acc[q].x = fmaf(w1, o[i + 1][q].x, fmaf(w0, o[i][q].x, acc[q].x));
            acc[q].y = fmaf(w1, o[i + 1][q].y, fmaf(w0, o[i][q].y, acc[q].y));
            acc[q].z = fmaf(w1, o[i + 1][q].z, fmaf(w0, o[i][q].z, acc[q].z));
            acc[q].w = fmaf(w1, o[i + 1][q].w, fmaf(w0, o[i][q].w, acc[q].w));
          }
        }
      }
    }
    const float inv = wsum != 0.f ? 1.f / wsum : 0.f;  // a NaN stays one
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
      const float4 r = make_float4(acc[q].x * inv, acc[q].y * inv, acc[q].z * inv, acc[q].w * inv);
      const int64_t at = (out_row0 + row) * kDv + d + 128 * q;
      if (a.o_bf16) {
        const __nv_bfloat162 x = __floats2bfloat162_rn(r.x, r.y), y = __floats2bfloat162_rn(r.z, r.w);
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o_part) + at) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
      } else {
        *reinterpret_cast<float4*>(static_cast<float*>(a.o_part) + at) = r;
      }
    }
    if (d == 0) {  // lane 0 of the row's first 128 dims
      const float lse2 = wsum != 0.f ? m + log2f(wsum) : -INFINITY;
      a.lse_part[out_row0 + row] = a.base2 ? lse2 : lse2 * kLn2;
    }
  }
}
// ---------------------------------------------------------------------------- host side
struct Plan {
  int Rg, ngroups, V, nts, nraw = 0, box_rows;
  size_t smem;
  size_t ws_start_bytes, ws_piece_o_bytes, ws_piece_lse_bytes, ws_total;
};

// The arguments of a partial-decode entry point (all but the workspace).
struct DecodeCall {
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
  void* o_part;
  int32_t o_part_dtype;
  float* lse_part;
  int32_t* status;
  void* stream;
};

int sm_count_current() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return n;
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// A main kernel's launch limits: its dynamic shared-memory limit per device, and
// the 2-CTA clusters of it that can be resident at once (both CTAs of a cluster
// share a GPC).  The counts are cached per device and shared-memory size (a
// workload uses one or two sizes); guarded by a mutex, since one host thread per
// GPU may plan at once.
class PairKernel {
 public:
  PairKernel(const void* fn, int threads) : fn_(fn), threads_(threads) {}
  bool ensure_smem(size_t smem) { return limit_.ensure(fn_, smem); }
  int max_active_clusters(size_t smem) {
    const int dev = current_device();
    if (dev < 0) return 0;
    {
      std::lock_guard<std::mutex> lock(m_);
      for (const Entry& e : cache_[dev])
        if (e.smem == smem && e.clusters > 0) return e.clusters;
    }
    if (!ensure_smem(smem)) return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * 512, 1, 1);
    cfg.blockDim = dim3(threads_, 1, 1);
    cfg.dynamicSmemBytes = smem;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, fn_, &cfg) != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
    if (n > 0) {
      std::lock_guard<std::mutex> lock(m_);
      Entry* slot = &cache_[dev][0];
      for (Entry& e : cache_[dev])
        if (e.clusters == 0 || e.smem == smem) {
          slot = &e;
          break;
        }
      *slot = Entry{smem, n};
    }
    return n;
  }

 private:
  struct Entry {
    size_t smem;
    int clusters;
  };
  static constexpr int kEntries = 8;
  const void* fn_;
  int threads_;
  SmemLimit limit_;
  std::mutex m_;
  Entry cache_[kMaxDevices][kEntries] = {};
};

// Row groups: at most 128 query rows each, as equal as multiples of 16 allow.
void plan_groups(int q_len, int H, Plan* p) {
  const int R_total = q_len * H;
  p->ngroups = (R_total + kMaxGroupRows - 1) / kMaxGroupRows;
  const int per = (R_total + p->ngroups - 1) / p->ngroups;
  p->Rg = ((per + 15) / 16) * 16;
}

// Copy boxes and workspace of a plan whose ranges are set.
void plan_workspace(const dcp_layout_t* layout, int n_held, int B, int R_total, Plan* p) {
  const int P = layout->page_size;
  p->box_rows = P >= kTile ? kTile : P;
  const int64_t U = (int64_t)B * n_held;
  p->ws_start_bytes = align256((size_t)(U + 1) * 4);
  // With one range per row group no unit is cut, so no piece is ever written.
  p->ws_piece_o_bytes = p->V > 1 ? align256((size_t)2 * p->V * R_total * kDv * 4) : 0;
  p->ws_piece_lse_bytes = p->V > 1 ? align256((size_t)2 * p->V * R_total * 4) : 0;
  p->ws_total = p->ws_start_bytes + p->ws_piece_o_bytes + p->ws_piece_lse_bytes;
}

// Stream-K ranges and workspace of a plan whose groups and shared memory are set.
bool plan_ranges(const dcp_layout_t* layout, int n_held, int B, int q_len, int H, PairKernel& kernel, Plan* p) {
  const int R_total = q_len * H;
  const int sms = sm_count_current();
  if (sms <= 0) return false;
  p->V = (sms / 2) / p->ngroups;  // ranges: one 2-CTA cluster per (range, row group)
  if (p->V < 1) p->V = 1;
  const int clusters = kernel.max_active_clusters(p->smem);
  if (clusters > 0) {
    // V ranges per row group.  One wave of V0 = clusters / ngroups ranges is the
    // default; when that leaves many clusters idle (ngroups not much below the
    // cluster count, e.g. a chunked extend's many row groups), a larger V run
    // in several waves finishes sooner: the time is waves / V of one group's
    // whole sequence.  A larger V must gain 5 % to pay for its cut units.
    const int V0 = clusters / p->ngroups > 1 ? clusters / p->ngroups : 1;
    auto cost = [&](int Vc) {
      return (double)(((int64_t)Vc * p->ngroups + clusters - 1) / clusters) / Vc;
    };
    int best = V0;
    for (int Vc = V0 + 1; Vc <= 8; ++Vc)
      if (cost(Vc) < 0.95 * cost(best)) best = Vc;
    p->V = best;
  }
  plan_workspace(layout, n_held, B, R_total, p);
  return true;
}

// bf16 [rows, 576] row-major, boxes of [box_rows, 64] with 128-byte swizzle, or
// (half = true) boxes of [box_rows, 32] with 64-byte swizzle
bool make_tmap(CUtensorMap* m, const void* base, uint64_t rows, uint32_t box_rows, bool half = false) {
  auto enc = tmap_encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)kDk, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)kDk * 2};
  cuuint32_t box[2] = {(cuuint32_t)(half ? kRopeHalf : kChunkDims), box_rows};
  cuuint32_t es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, half ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows of a unit that its row of the block table can hold.
int64_t table_rows(const dcp_layout_t* layout, int64_t max_pages) {
  return std::min(std::min(max_pages, kMaxUnitRows) * layout->page_size, kMaxUnitRows);
}

bool page_size_ok(int P) { return P >= 8 && P % 8 == 0 && (P % kTile == 0 || kTile % P == 0); }

// Host checks of a partial decode's arguments (all but the workspace).
int32_t check_decode_args(const DecodeCall& c) {
  if (!layout_ok(c.layout) || c.shard_begin < 0 || c.shard_end > c.layout->n_shards || c.shard_begin >= c.shard_end)
    return DCP_ERR_INVALID;
  if (c.B < 1 || c.q_len < 1 || c.H < 1 || (int64_t)c.q_len * c.H > kMaxQueryRows) return DCP_ERR_INVALID;
  if (c.pool_pages < 1 || c.max_pages < 1 || c.bt_stride < c.max_pages) return DCP_ERR_INVALID;
  if (!c.q || !c.arena || !c.block_table || !c.seq_lens || !c.o_part || !c.lse_part) return DCP_ERR_INVALID;
  if (c.o_part_dtype != DCP_F32 && c.o_part_dtype != DCP_BF16) return DCP_ERR_INVALID;
  if (c.lse_base != DCP_LSE_BASE_E && c.lse_base != DCP_LSE_BASE_2) return DCP_ERR_INVALID;
  if (!(c.scale > 0.f) || !(c.scale < INFINITY)) return DCP_ERR_INVALID;
  if ((reinterpret_cast<uintptr_t>(c.q) | reinterpret_cast<uintptr_t>(c.arena) |
       reinterpret_cast<uintptr_t>(c.o_part)) & 15)
    return DCP_ERR_INVALID;
  if (!page_size_ok(c.layout->page_size)) return DCP_ERR_UNSUPPORTED;
  const int64_t pool_rows = c.pool_pages * c.layout->page_size;
  const int64_t n_held = c.shard_end - c.shard_begin;
  if (n_held * pool_rows >= INT32_MAX || (int64_t)c.B * c.q_len * c.H >= INT32_MAX ||
      (int64_t)c.B * n_held >= INT32_MAX / 2)
    return DCP_ERR_UNSUPPORTED;
  // The lengths are only known on the device: with every unit as long as its table row, the
  // planner's sums of tiles stay in 32 bits.
  const int64_t unit_tiles = (table_rows(c.layout, c.max_pages) + kTile - 1) / kTile;
  if ((int64_t)c.B * n_held * unit_tiles >= INT32_MAX) return DCP_ERR_UNSUPPORTED;
  return DCP_OK;
}

// Arguments of a workspace-size query.
bool size_args_ok(const dcp_layout_t* layout, int32_t shard_begin, int32_t shard_end, int32_t B, int32_t q_len,
                  int32_t H) {
  return layout_ok(layout) && shard_begin >= 0 && shard_end <= layout->n_shards && shard_begin < shard_end && B >= 1 &&
         q_len >= 1 && H >= 1 && (int64_t)q_len * H <= kMaxQueryRows;
}

// A caller's workspace for a plan.
int32_t check_workspace(const Plan& p, const void* workspace, size_t bytes) {
  if (!workspace || bytes < p.ws_total) return DCP_ERR_WORKSPACE;
  return (reinterpret_cast<uintptr_t>(workspace) & 255) ? DCP_ERR_INVALID : DCP_OK;
}

// Device arguments of a checked call on a workspace of at least p.ws_total bytes
// (256-byte aligned).
TcArgs device_args(const Plan& p, const DecodeCall& c, void* workspace) {
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  TcArgs a;
  a.L = to_layout(c.layout);
  a.shard_begin = c.shard_begin;
  a.n_held = c.shard_end - c.shard_begin;
  a.B = c.B; a.q_len = c.q_len; a.H = c.H; a.R_total = c.q_len * c.H;
  a.Rg = p.Rg; a.ngroups = p.ngroups; a.V = p.V; a.nts = p.nts; a.nraw = p.nraw; a.box_rows = p.box_rows;
  a.q = static_cast<const __nv_bfloat16*>(c.q);
  a.pool_rows = c.pool_pages * c.layout->page_size; a.pool_pages = c.pool_pages;
  a.max_rows = table_rows(c.layout, c.max_pages);
  a.bt = c.block_table; a.bt_stride = c.bt_stride; a.max_pages = c.max_pages;
  a.seq_lens = c.seq_lens;
  a.scale_log2 = c.scale * kLog2e;
  a.base2 = c.lse_base == DCP_LSE_BASE_2;
  a.o_part = c.o_part; a.o_bf16 = c.o_part_dtype == DCP_BF16;
  a.lse_part = c.lse_part;
  a.tile_start = reinterpret_cast<const int32_t*>(ws);
  a.piece_o = reinterpret_cast<float*>(ws + p.ws_start_bytes);
  a.piece_lse = reinterpret_cast<float*>(ws + p.ws_start_bytes + p.ws_piece_o_bytes);
  a.status = c.status;
  return a;
}

// The three launches of one partial decode: planner, the main kernel (enqueued by
// launch_main with the given configuration) and the merge of cut units.
template <class LaunchMain>
int32_t launch_decode(const Plan& p, const TcArgs& a, int threads, void* stream, LaunchMain launch_main) {
  cudaStream_t st = as_stream(stream);
  plan_kernel<<<1, 1024, 0, st>>>(a, const_cast<int32_t*>(a.tile_start), a.B * a.n_held);
  // The partial kernel and the fixup are programmatic dependent launches: each
  // grid may be scheduled while the one before it finishes, and waits
  // (griddepcontrol.wait) before it reads anything that one wrote.
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)(2 * p.V * p.ngroups));
  lc.blockDim = dim3(threads);
  lc.dynamicSmemBytes = p.smem;
  lc.stream = st;
  lc.attrs = pdl;
  lc.numAttrs = 1;
  if (launch_main(lc) != cudaSuccess) return DCP_ERR_CUDA;
  // Cut units need their pieces merged: one block column per range boundary, blocks
  // looping over chunks of rows.  With one range per row group nothing is cut and no
  // fixup runs.
  if (p.V > 1) {
    const bool few = a.R_total <= kFixupFewRows;
    const int items = a.R_total * (few ? 2 : 1);
    const unsigned fix_y = (unsigned)std::min((items + kFixupWarps - 1) / kFixupWarps, 12);
    cudaLaunchConfig_t lf = {};
    lf.gridDim = dim3((unsigned)(p.V - 1), fix_y);
    lf.blockDim = dim3(kFixupThreads);
    lf.stream = st;
    lf.attrs = pdl;
    lf.numAttrs = 1;
    if (cudaLaunchKernelEx(&lf, few ? fixup_kernel<2> : fixup_kernel<4>, a) != cudaSuccess) return DCP_ERR_CUDA;
    return launch_status(3);
  }
  return launch_status(2);
}

}  // namespace
