// dcp_tables.cu — block tables, the free-page list and the new tokens' slots,
// built on the device from request lengths.
//
// Sources: SGLang "Decode context parallelism", "Virtual KV layout" (a widened
// page of N * P positions is one physical page on every shard, so a request of x
// positions holds ceil(x / (N P)) pages of one table shared by all shards);
// "PCP / DCP：计算、KV 布局与块轮转", section "KV cache 管理" (page tables and
// slots); the slot formulas are dcp_slot_map's.
//
// One block scans the requests (new tokens, pages to take, pages to give back),
// then spreads the pages and, for a short list, the tokens over its threads: each
// finds its request by bisection of the prefix sums in shared memory.  A long
// list of tokens goes to a second launch with a thread per token, which bisects
// cu_tokens.  Everything is integer and every entry has one writer, so the result
// does not depend on any order.  Latency-bound: 128 requests, 4 tokens each, take
// 5 us in a captured graph, most of it the block's scan and one dependent load after
// another; a long list of tokens adds a launch that writes 32 bytes a token.
#include "dcp_internal.cuh"

using namespace dcp;

namespace {

constexpr int kPlanThreads = 1024;
// Longest list the scanning block writes itself.  Two calls, growing and giving back,
// take with 256 entries 9.9 us written here and 12.1 by the second launch; with 2048
// 13.4 and 13.7; with 4096 17.0 and 14.0; with 16384 40.9 and 14.0.
constexpr int64_t kInlineTokens = 2048;

struct TableArgs {
  Layout L;
  int32_t B;
  int64_t* seq_lens;
  const int64_t* new_lens;
  int32_t* bt;
  int64_t bt_stride, max_pages;
  int32_t* ring;      // free_pages: a ring of pool_pages entries
  int64_t* state;     // {head, count}
  int64_t pool_pages;
  int64_t T;          // entries of the token arrays (0: no list)
  int64_t* pos;
  int32_t* req;
  int32_t* owner;
  int64_t* row;
  int64_t* slot;
  int64_t* cu;
  int32_t* status;
};

struct Counts {
  int64_t tokens, take, give;
};

// Request b's lengths and their pages before and after.
struct Request {
  int64_t old_len, new_len, old_pages, new_pages;
};

__device__ __forceinline__ Counts operator+(const Counts& a, const Counts& b) {
  return Counts{a.tokens + b.tokens, a.take + b.take, a.give + b.give};
}

// Pages of x >= 0 positions, `span` of which share one (32-bit division where it does).
__device__ __forceinline__ int64_t pages_of(int64_t x, int64_t span) {
  if (x <= INT32_MAX && span <= INT32_MAX) return (int64_t)(((uint32_t)x + (uint32_t)span - 1) / (uint32_t)span);
  return x / span + (x % span != 0);
}

// What request b needs for its new length; *bad gets the status bits of a length
// that cannot be.
__device__ __forceinline__ Counts needs(const TableArgs& a, int32_t b, Request& q, int& bad) {
  q = Request{a.seq_lens[b], a.new_lens[b], 0, 0};
  // (a length above 2^62 / B is none either: sums of B lengths stay in 64 bits)
  const int64_t most = (int64_t(1) << 62) / a.B;
  if (q.old_len < 0 || q.new_len < 0 || q.old_len > most || q.new_len > most) {
    bad |= DCP_STATUS_BAD_LENGTH;
    return Counts{0, 0, 0};
  }
  const int64_t span = a.L.N * a.L.P;
  q.old_pages = pages_of(q.old_len, span);
  q.new_pages = pages_of(q.new_len, span);
  if (q.old_pages > a.max_pages || q.new_pages > a.max_pages) {
    bad |= DCP_STATUS_BAD_PAGE_INDEX;
    return Counts{0, 0, 0};
  }
  return Counts{max(q.new_len - q.old_len, (int64_t)0), max(q.new_pages - q.old_pages, (int64_t)0),
                max(q.old_pages - q.new_pages, (int64_t)0)};
}

__device__ __forceinline__ Counts warp_scan(Counts x, int lane) {
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const Counts y{__shfl_up_sync(0xffffffffu, x.tokens, s), __shfl_up_sync(0xffffffffu, x.take, s),
                   __shfl_up_sync(0xffffffffu, x.give, s)};
    if (lane >= s) x = x + y;
  }
  return x;
}

// Inclusive scan over the block's threads; *total gets the sum.
__device__ __forceinline__ Counts block_scan(Counts x, Counts* sums, Counts* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  x = warp_scan(x, lane);
  __syncthreads();  // sums may still be read from the scan before
  if (lane == 31) sums[w] = x;
  __syncthreads();
  if (w == 0) sums[lane] = warp_scan(sums[lane], lane);
  __syncthreads();
  *total = sums[kPlanThreads / 32 - 1];
  return w > 0 ? sums[w - 1] + x : x;
}

// Largest k in [0, n) with start[k] <= x, for start[0] <= x: of equal entries the
// last, so the one that is not empty.
template <class Int>
__device__ __forceinline__ int32_t find(const Int* start, int32_t n, int64_t x) {
  int32_t lo = 0, hi = n;
  while (hi - lo > 1) {
    const int32_t m = (lo + hi) >> 1;
    if ((int64_t)start[m] <= x) lo = m; else hi = m;
  }
  return lo;
}

// Entry t of the token list: position p of request b (p = b = -1: no token).
__device__ __forceinline__ void write_token(const TableArgs& a, int64_t t, int64_t p, int32_t b) {
  a.pos[t] = p;
  a.req[t] = b;
  if (!a.owner && !a.row && !a.slot) return;
  int64_t own = -1, row = -1, slot = -1;
  if (p >= 0) {
    int64_t pidx;
    if (p < INT32_MAX) {
      const int32_t p32 = (int32_t)p, I = (int32_t)a.L.I, N = (int32_t)a.L.N, blk = p32 / I;
      own = blk % N;
      row = (int64_t)(blk / N) * I + p32 % I;
      pidx = (int32_t)row / (int32_t)a.L.P;
    } else {
      own = owner_of(p, a.L);
      row = local_row_of(p, a.L);
      pidx = row / a.L.P;
    }
    if (a.slot) {
      // pidx < pages of the new length <= max_pages
      const int64_t page = a.bt[(int64_t)b * a.bt_stride + pidx];
      if (page < 0 || page >= a.pool_pages)
        flag(a.status, DCP_STATUS_BAD_PAGE_ID);
      else
        slot = page * a.L.P + (row - pidx * a.L.P);
    }
  }
  if (a.owner) a.owner[t] = (int32_t)own;
  if (a.row) a.row[t] = row;
  if (a.slot) a.slot[t] = slot;
}

__global__ void __launch_bounds__(kPlanThreads) block_tables_kernel(TableArgs a) {
  __shared__ Counts sums[32];
  __shared__ int64_t tok_s[kPlanThreads];  // exclusive prefix sums of the chunk's requests
  __shared__ int32_t take_s[kPlanThreads], give_s[kPlanThreads];
  __shared__ int64_t len_s[kPlanThreads];  // their old lengths
  __shared__ int64_t keep_s[kPlanThreads];  // the smaller of their old and new pages
  const int tid = threadIdx.x;
  const int64_t head = a.state[0], count = a.state[1], cap = a.pool_pages;
  int bad = 0;
  // Totals first: the call happens as a whole or not at all.  (A single chunk of
  // requests is not looked at again afterwards.)
  Counts need{0, 0, 0}, x{0, 0, 0}, end{0, 0, 0}, part{0, 0, 0};
  Request q{0, 0, 0, 0};
  for (int32_t base = 0; base < a.B; base += kPlanThreads) {
    const int32_t b = base + tid;
    x = b < a.B ? needs(a, b, q, bad) : Counts{0, 0, 0};
    end = block_scan(x, sums, &part);
    need = need + part;
  }
  if (head < 0 || head >= cap || count < 0 || count > cap || need.give > cap - count)
    bad |= DCP_STATUS_BAD_POOL;
  else if (need.take > count)
    bad |= DCP_STATUS_NO_PAGES;
  if (a.pos && need.tokens > a.T) bad |= DCP_STATUS_TOO_MANY_TOKENS;
  const bool ok = !__syncthreads_or(bad);
  if (bad) flag(a.status, bad);
  Counts done{0, 0, 0};
  for (int32_t base = 0; base < a.B; base += kPlanThreads) {
    const int32_t b = base + tid;
    if (!ok) {
      x = end = part = Counts{0, 0, 0};
    } else if (a.B > kPlanThreads) {
      x = b < a.B ? needs(a, b, q, bad) : Counts{0, 0, 0};
      end = block_scan(x, sums, &part);
    }
    tok_s[tid] = done.tokens + end.tokens - x.tokens;
    take_s[tid] = (int32_t)(end.take - x.take);   // at most pool_pages
    give_s[tid] = (int32_t)(end.give - x.give);
    len_s[tid] = q.old_len;
    keep_s[tid] = min(q.old_pages, q.new_pages);
    if (b < a.B) {
      a.cu[b + 1] = done.tokens + end.tokens;
      if (ok) a.seq_lens[b] = q.new_len;
    }
    __syncthreads();
    const int32_t here = min(kPlanThreads, a.B - base);
    // The ring's entries that are taken hold free pages and those written with
    // returned ones do not, so the two never meet.
    for (int64_t i = tid; i < part.take; i += kPlanThreads) {
      const int32_t k = find(take_s, here, i);
      const int64_t pidx = keep_s[k] + (i - take_s[k]);
      int64_t at = head + done.take + i;
      if (at >= cap) at -= cap;
      a.bt[(int64_t)(base + k) * a.bt_stride + pidx] = a.ring[at];
    }
    for (int64_t i = tid; i < part.give; i += kPlanThreads) {
      const int32_t k = find(give_s, here, i);
      const int64_t pidx = keep_s[k] + (i - give_s[k]);
      int32_t* entry = a.bt + (int64_t)(base + k) * a.bt_stride + pidx;
      const int32_t page = *entry;
      if (page < 0 || page >= cap) flag(a.status, DCP_STATUS_BAD_PAGE_ID);
      int64_t at = head + count + done.give + i;   // below 3 cap
      while (at >= cap) at -= cap;
      a.ring[at] = page;
      *entry = -1;
    }
    if (a.pos && a.T <= kInlineTokens) {
      __syncthreads();  // the pages just taken
      for (int64_t t = done.tokens + tid; t < done.tokens + part.tokens; t += kPlanThreads) {
        const int32_t k = find(tok_s, here, t);
        write_token(a, t, len_s[k] + (t - tok_s[k]), base + k);
      }
    }
    done = done + part;
    __syncthreads();  // the shared arrays are reused
  }
  if (a.pos && a.T <= kInlineTokens)
    for (int64_t t = done.tokens + tid; t < a.T; t += kPlanThreads) write_token(a, t, -1, -1);
  if (tid == 0) {
    a.cu[0] = 0;
    if (ok) {
      int64_t h = head + done.take;
      if (h >= cap) h -= cap;
      a.state[0] = h;
      a.state[1] = count - done.take + done.give;
    }
  }
}

// A long token list: thread t writes entry t, after block_tables_kernel.
__global__ void __launch_bounds__(256) token_list_kernel(TableArgs a) {
  const int64_t t = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  if (t >= a.T) return;
  if (t >= a.cu[a.B]) {
    write_token(a, t, -1, -1);
    return;
  }
  const int32_t b = find(a.cu, a.B, t);
  write_token(a, t, a.seq_lens[b] - (a.cu[b + 1] - t), b);
}

}  // namespace

extern "C" int32_t dcp_block_tables(const dcp_layout_t* layout, int32_t B, int64_t* seq_lens, const int64_t* new_lens,
                                    int32_t* block_table, int64_t bt_stride, int64_t max_pages, int32_t* free_pages,
                                    int64_t* free_state, int64_t pool_pages, int64_t T, int64_t* pos, int32_t* req,
                                    int32_t* owner, int64_t* row, int64_t* slot, int64_t* cu_tokens, int32_t* status,
                                    void* stream) {
  if (!layout_ok(layout) || B < 1 || max_pages < 1 || bt_stride < max_pages || pool_pages < 1 ||
      pool_pages > INT32_MAX || T < 0)
    return DCP_ERR_INVALID;
  if (!seq_lens || !new_lens || !block_table || !free_pages || !free_state || !cu_tokens || !status)
    return DCP_ERR_INVALID;
  if ((pos == nullptr) != (req == nullptr) || (!pos && (owner || row || slot))) return DCP_ERR_INVALID;
  if (seq_lens == new_lens) return DCP_ERR_INVALID;
  const int64_t blocks = (T + 255) / 256;
  if (blocks > INT32_MAX) return DCP_ERR_UNSUPPORTED;
  const TableArgs a{to_layout(layout), B, seq_lens, new_lens, block_table, bt_stride, max_pages, free_pages,
                    free_state, pool_pages, T, pos, req, owner, row, slot, cu_tokens, status};
  block_tables_kernel<<<1, kPlanThreads, 0, as_stream(stream)>>>(a);
  if (!pos || T <= kInlineTokens) return launch_status();
  const int32_t rc = launch_status();
  if (rc != DCP_OK) return rc;
  token_list_kernel<<<(unsigned)blocks, 256, 0, as_stream(stream)>>>(a);
  return launch_status();
}
