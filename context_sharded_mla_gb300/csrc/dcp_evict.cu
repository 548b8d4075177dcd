// dcp_evict.cu — a cache made shorter by what its rows weigh: which rows of each shard
// stay, and their move to the front of the shard, in place.
//
// Each shard keeps count_r(new length) of its own rows ("PCP / DCP：计算、KV 布局与块
// 轮转", section 6: local_len), so that no row leaves its shard and the layout's count
// rule holds for what is left; kept rows stay in order.
//
// select_kernel: one cluster of CTAs for a (request, shard) unit.  The k-th largest
// weight of the rows that compete is found digit by digit, 8 bits of an order-preserving
// integer at a time: histograms in shared memory, one copy a lane, so that the lanes of a
// warp never meet in a bank however alike their weights are (weights of one
// magnitude share their first digit); the CTAs add theirs up through distributed shared
// memory.  Rows are then written in order: counts a warp, prefix sums, ballots.  Only
// whole numbers are added, so the result depends on no order.  It reads the weights six
// times, five of them from L1 or L2.
//
// compact_kernel: row i <- row kept[i] >= i.  Writing row i is safe once the rows up to
// i have been read: a later row j > i reads kept[j] >= j.  So a cluster walks a unit in
// windows, reads a window (bulk copies into a ring of slots in shared memory, several
// windows ahead), and writes it when every CTA of the cluster has its part of it.
// Memory-bound: 2 * 1152 (or 416) bytes a row; a warp issues everything.
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
  const uint32_t u = __float_as_uint(w);
  if (w != w) return 0xFFFFFFFFu;
  if (w == 0.f) return 0x80000000u;
  return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
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

__global__ void __launch_bounds__(kSelThreads) select_kernel(SelectArgs a) {
  __shared__ uint32_t hist[kBins * 32];
  __shared__ uint32_t total[kDigits][kBins];  // this CTA's counts of each digit's bins, read by the cluster
  __shared__ uint32_t all[kBins];
  __shared__ uint32_t pick_s[2];              // chosen bin, rows still wanted of it
  __shared__ uint32_t warp_gt[kSelWarps], warp_eq[kSelWarps];
  __shared__ uint32_t cta_n[2];               // rows above and at the limit
  const uint32_t rank = cluster_ctarank(), nranks = cluster_nctarank();
  const int64_t u = blockIdx.x / nranks;
  const int rs = (int)(u / a.B), b = (int)(u % a.B);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t S = a.seq_lens[b], M = a.new_lens[b];
  const int64_t r = a.shard_begin + rs;
  const int64_t m = M > 0 ? count_of(r, M, a.L) : 0;
  const int64_t n = S > 0 ? count_of(r, S, a.L) : 0;
  int32_t* kept = a.kept + u * a.kept_stride;
  if (M < 0 || M > S || n > a.w_stride || m > a.kept_stride) {  // refused: the whole cluster leaves
    if (tid == 0 && rank == 0) flag(a.status, DCP_STATUS_BAD_LENGTH);
    const int64_t e = m < a.kept_stride ? m : a.kept_stride;
    for (int64_t i = rank * kSelThreads + tid; i < e; i += nranks * kSelThreads) kept[i] = -1;
    return;
  }
  // rows [0, lo) are sinks, [hi, n) recent ones, those between compete
  const int64_t lo = count_of(r, a.sinks < S ? a.sinks : S, a.L);
  const int64_t zr = count_of(r, S > a.recent ? S - a.recent : 0, a.L);
  const int64_t hi = zr > lo ? zr : lo;
  const int64_t ns = lo < m ? lo : m;
  const int64_t nr = m - ns < n - hi ? m - ns : n - hi;
  const int64_t len = hi - lo;
  uint32_t want = (uint32_t)(m - ns - nr);  // of the rows between; rows of a unit fit 31 bits (w_stride)
  if (rank == 0)
    for (int64_t i = tid; i < ns; i += kSelThreads) kept[i] = (int32_t)i;
  if (rank == nranks - 1)
    for (int64_t i = tid; i < nr; i += kSelThreads) kept[m - nr + i] = (int32_t)(n - nr + i);
  if (want == 0) return;  // uniform over the cluster

  // this CTA's rows, and this warp's of them
  const int64_t per = ((len + nranks - 1) / nranks + 31) / 32 * 32;
  const int32_t c0 = (int32_t)(rank * per < len ? rank * per : len);
  const int32_t c1 = (int32_t)(c0 + per < len ? c0 + per : len);
  const float* w = a.weights + u * a.w_stride + lo;
  uint32_t prefix = 0;
#pragma unroll 1
  for (int d = 0; d < kDigits; ++d) {
    const int shift = 24 - 8 * d;
    for (int i = tid; i < kBins * 32; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    const uint32_t mask = d ? 0xFFFFFFFFu << (shift + 8) : 0u;
#pragma unroll 4
    for (int32_t i = c0 + tid; i < c1; i += kSelThreads) {
      const uint32_t k = order_key(w[i]);
      if ((k & mask) == prefix) atomicAdd(&hist[((k >> shift) & 255u) * 32 + lane], 1u);
    }
    __syncthreads();
    {
      const int bin = tid >> 1;
      uint32_t s = 0;
#pragma unroll
      for (int k = 0; k < 16; ++k) s += hist[bin * 32 + 16 * (tid & 1) + ((k + (tid >> 1)) & 15)];
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      if (!(tid & 1)) total[d][bin] = s;
    }
    if (nranks > 1) cluster_sync(); else __syncthreads();
    if (tid < kBins) {
      uint32_t s = 0;
      for (uint32_t c = 0; c < nranks; ++c)
        s += nranks > 1 ? ld_cluster_u32(mapa_shared(smem_u32(&total[d][tid]), c)) : total[d][tid];
      all[tid] = s;
    }
    __syncthreads();
    if (warp == 0) {  // the bin that holds the want-th largest: counts from the top, 8 bins a lane
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
            pick_s[0] = 255 - 8 * lane - k;
            pick_s[1] = want - before;
          }
          before += c[k];
        }
      }
    }
    __syncthreads();
    prefix |= pick_s[0] << shift;
    want = pick_s[1];
  }
  // rows above the limit `prefix` stay, and the first `want` of those at it
  const int32_t perw = ((c1 - c0 + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
  const int32_t w0 = min(c0 + warp * perw, c1), w1 = min(w0 + perw, c1);
  int gt = 0, eq = 0;
#pragma unroll 4
  for (int32_t i = w0 + lane; i < w1; i += 32) {
    const uint32_t k = order_key(w[i]);
    gt += k > prefix;
    eq += k == prefix;
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
    cta_n[0] = sg;
    cta_n[1] = se;
  }
  uint32_t gt0 = 0, eq0 = 0;  // rows above and at the limit before this warp's
  if (nranks > 1) {
    cluster_sync();
    for (uint32_t c = 0; c < rank; ++c) {
      gt0 += ld_cluster_u32(mapa_shared(smem_u32(&cta_n[0]), c));
      eq0 += ld_cluster_u32(mapa_shared(smem_u32(&cta_n[1]), c));
    }
  }
  for (int i = 0; i < warp; ++i) {
    gt0 += warp_gt[i];
    eq0 += warp_eq[i];
  }
  const uint32_t below = (1u << lane) - 1;
  for (int32_t i = w0; i < w1; i += 32) {
    const bool in = i + lane < w1;
    const uint32_t k = in ? order_key(w[i + lane]) : 0u;
    const uint32_t bg = __ballot_sync(0xffffffffu, in && k > prefix), be = __ballot_sync(0xffffffffu, in && k == prefix);
    const uint32_t at_eq = eq0 + __popc(be & below);
    if (in && (k > prefix || (k == prefix && at_eq < want)))
      kept[ns + gt0 + __popc(bg & below) + (at_eq < want ? at_eq : want)] = (int32_t)(lo + i + lane);
    gt0 += __popc(bg);
    eq0 += __popc(be);
  }
  if (nranks > 1) cluster_sync();  // no CTA leaves while its counts are read
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

// Rows a window and windows a ring: about 108 KB a CTA, two CTAs an SM.
template <int kRowBytes>
struct Ring {
  static constexpr int kRows = kRowBytes > 1024 ? 16 : 32;
  static constexpr int kWindows = kRowBytes > 1024 ? 6 : 8;
  static constexpr int kSlotBytes = kRows * kRowBytes;
  static constexpr int kSmem = kWindows * kSlotBytes;
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

template <int kRowBytes>
__global__ void __launch_bounds__(32) compact_kernel(CompactArgs a) {
  using R = Ring<kRowBytes>;
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ uint64_t full[R::kWindows];
  __shared__ float w_s[R::kWindows][R::kRows];
  __shared__ int abort_w;
  volatile int* abort_s = &abort_w;
  const uint32_t rank = cluster_ctarank();
  uint32_t nranks;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(nranks));
  const int64_t u = blockIdx.x / nranks;
  const int rs = (int)(u / a.B), b = (int)(u % a.B), lane = threadIdx.x;
  const int64_t M = a.new_lens[b];
  const int64_t m64 = M > 0 ? count_of(a.shard_begin + rs, M, a.L) : 0;
  if (M < 0 || m64 > a.kept_stride) {  // uniform over the cluster
    if (lane == 0 && rank == 0) flag(a.status, DCP_STATUS_BAD_LENGTH);
    return;
  }
  const int32_t m = (int32_t)m64;
  if (m == 0) return;
  if (lane == 0) {
    *abort_s = 0;
    for (int i = 0; i < R::kWindows; ++i) mbar_init(&full[i], 33);  // the byte count, and every lane's weight
    fence_barrier_init();
  }
  __syncwarp();
  const int32_t* kept = a.kept + u * a.kept_stride;
  const int32_t* bt = a.bt + (int64_t)b * a.bt_stride;
  float* wts = a.weights ? a.weights + u * a.w_stride : nullptr;
  unsigned char* pool = a.arena + rs * a.pool_pages * a.L.P * kRowBytes;
  const int32_t P = (int32_t)a.L.P;
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
    if (k / P >= a.max_pages || (wts && k >= a.w_stride)) {
      flag(a.status, DCP_STATUS_BAD_PAGE_INDEX);
      return Pages{-1, 0, 0};
    }
    return Pages{k, __ldg(bt + k / P), __ldg(bt + (int32_t)i / P)};
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
      bulk_load(ring + s * R::kSlotBytes + lane * kRowBytes, pool + ((int64_t)pg.src * P + pg.from % P) * kRowBytes,
                kRowBytes, &full[s]);
      if (wts) copy4_async(smem_u32(&w_s[s][lane]), wts + pg.from);
    }
    copies_arrive(&full[s]);
    return live ? pool + ((int64_t)pg.dst * P + i % P) * kRowBytes : nullptr;
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
  bool ok = true;
  for (int32_t x0 = 0; x0 < nwin; x0 += R::kWindows) {
#pragma unroll
    for (int s = 0; s < R::kWindows; ++s) {
      const int32_t x = x0 + s;
      if (x >= nwin) break;
      if (ok) {
        bool here = mbar_wait(&full[s], (uint32_t)(x / R::kWindows) & 1u, abort_s);
        ok = __all_sync(0xffffffffu, here);
      }
      if (nranks > 1) cluster_sync();  // after a wait that ran out too: the others count on it
      if (ok) {
        if (dst[s]) {
          bulk_store(dst[s], smem_u32(ring) + s * R::kSlotBytes + lane * kRowBytes, kRowBytes);
          if (wts) wts[row_at(x)] = w_s[s][lane];
        }
        bulk_commit();
        if (x + kAhead < nwin) {
          bulk_wait_read<2>();  // window x - 2 has left the slot that is filled next
          dst[(s + kAhead) % R::kWindows] = feed(x + kAhead);
        }
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

SmemLimit g_compact_bf16, g_compact_q4;

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

template <int kRowBytes>
int32_t compact(SmemLimit& limit, const dcp_layout_t* layout, int32_t shard_begin, int32_t shard_end,
                const int32_t* kept, int64_t kept_stride, int32_t B, const int64_t* new_lens,
                const int32_t* block_table, int64_t bt_stride, int64_t max_pages, void* arena, int64_t pool_pages,
                float* weights, int64_t w_stride, int32_t* status, void* stream) {
  if (!shards_ok(layout, shard_begin, shard_end, B) || kept_stride < 0 || max_pages < 1 || bt_stride < max_pages ||
      pool_pages < 1 || (weights && w_stride < 1))
    return DCP_ERR_INVALID;
  if (!new_lens || !block_table || !arena || (kept_stride && !kept) || (reinterpret_cast<uintptr_t>(arena) & 15))
    return DCP_ERR_INVALID;
  if (kept_stride == 0) return DCP_OK;
  if (kept_stride > INT32_MAX - 1024) return DCP_ERR_UNSUPPORTED;  // kept entries are 32-bit rows
  using R = Ring<kRowBytes>;
  if (!limit.ensure(reinterpret_cast<const void*>(&compact_kernel<kRowBytes>), R::kSmem)) return DCP_ERR_CUDA;
  const CompactArgs a{to_layout(layout), shard_begin, shard_end - shard_begin, B, kept, kept_stride, new_lens,
                      block_table, bt_stride, max_pages, static_cast<unsigned char*>(arena), pool_pages, weights,
                      w_stride, status};
  const int64_t units = (int64_t)B * a.n_held;
  return launch_clusters(compact_kernel<kRowBytes>, units, cluster_of(units, kept_stride, 2 * R::kRows, 304), 32, R::kSmem,
                         stream, a);
}

}  // namespace

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
  return launch_clusters(select_kernel, units, cluster_of(units, w_stride, 2048, 608), kSelThreads, 0, stream, a);
}

extern "C" int32_t dcp_kv_compact(const dcp_layout_t* layout, int32_t shard_begin, int32_t shard_end,
                                  const int32_t* kept, int64_t kept_stride, int32_t B, const int64_t* new_lens,
                                  const int32_t* block_table, int64_t bt_stride, int64_t max_pages, void* arena,
                                  int64_t pool_pages, float* weights, int64_t w_stride, int32_t* status,
                                  void* stream) {
  return compact<kDk * 2>(g_compact_bf16, layout, shard_begin, shard_end, kept, kept_stride, B, new_lens, block_table,
                          bt_stride, max_pages, arena, pool_pages, weights, w_stride, status, stream);
}

extern "C" int32_t dcp_kv_compact_q4(const dcp_layout_t* layout, int32_t shard_begin, int32_t shard_end,
                                     const int32_t* kept, int64_t kept_stride, int32_t B, const int64_t* new_lens,
                                     const int32_t* block_table, int64_t bt_stride, int64_t max_pages, void* arena,
                                     int64_t pool_pages, float* weights, int64_t w_stride, int32_t* status,
                                     void* stream) {
  return compact<kQ4RowBytes>(g_compact_q4, layout, shard_begin, shard_end, kept, kept_stride, B, new_lens, block_table,
                              bt_stride, max_pages, arena, pool_pages, weights, w_stride, status, stream);
}
