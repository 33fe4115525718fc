// ivc_cache.cu — pages of the key/value cache behind the spliced sequence:
// taking, sharing, copying, compacting and giving them back.
//
// Each operation is a device plan and (fork, compact) a move of rows by that
// plan, as in the sequence assembly (ivc_assemble.cu): no length or page number
// is read on the host, so a call can be captured and replayed.
//
// The plan is one CTA. It first checks everything that the operation is going
// to touch, and only when all of it is sound changes the tables: a refused call
// leaves the cache as it was. Counts are integers and pages are handed out by
// prefix sums, so results do not depend on thread order; freed pages are
// collected as bits of a bitmap in shared memory (one bit per page, at most
// 128 KB), which both finds the last holder's release exactly once and lists
// the freed pages in ascending order.
#include <cuda_runtime.h>

#include "ivc_internal.h"
#include "ivc_ptx.cuh"

namespace ivc {
namespace {

constexpr int CA_THREADS = 1024;
constexpr int CA_WARPS = CA_THREADS / 32;
constexpr int CA_MAX_SEQS = 65536;
constexpr int CA_MAX_PAGES = 1 << 20;

// What the plan kernels keep in shared memory besides the page bitmap.
struct PlanShared {
  unsigned seen[CA_MAX_SEQS / 32];  // sequences named by this call
  int order[CA_THREADS];            // one pass of sequences: pages before this one's
  int need[CA_THREADS];             // pages it takes
  long long warp_sum[CA_WARPS];
  int bad;                          // DEV_* bits
};

// Exclusive sum over the CTA; every thread calls it. `total` gets the whole sum.
__device__ long long block_scan(long long v, long long* s_warp, long long& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long long incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    long long w = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long t = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += t;
    }
    s_warp[lane] = w;
  }
  __syncthreads();
  const long long before = warp > 0 ? s_warp[warp - 1] : 0;
  total = s_warp[CA_WARPS - 1];
  __syncthreads();
  return before + incl - v;
}

__device__ __forceinline__ int seq_of(const int32_t* seqs, int i) { return seqs ? seqs[i] : i; }

// Marks sequence s as named; 0, or DEV_BAD_CACHE when it is outside the cache,
// named before, or its length and pages do not fit together.
__device__ int claim_seq(const ivc_cache& c, PlanShared& sh, int s) {
  if (s < 0 || s >= c.max_seqs) return DEV_BAD_CACHE;
  const unsigned bit = 1u << (s & 31);
  if (atomicOr(&sh.seen[s >> 5], bit) & bit) return DEV_BAD_CACHE;
  return 0;
}
__device__ int seq_sound(const ivc_cache& c, int s) {
  const int np = c.n_pages[s], len = c.length[s];
  if (np < 0 || np > c.max_pages || len < 0) return DEV_BAD_CACHE;
  return static_cast<long long>(np) * c.page_tokens < len ? DEV_BAD_CACHE : 0;
}
__device__ __forceinline__ bool page_ok(const ivc_cache& c, int p) { return p >= 0 && p < c.pages; }

__device__ void plan_begin(const ivc_cache& c, PlanShared& sh) {
  for (int i = threadIdx.x; i < (c.max_seqs + 31) / 32; i += CA_THREADS) sh.seen[i] = 0;
  if (threadIdx.x == 0) {
    const int fc = *c.free_count;
    sh.bad = fc < 0 || fc > c.pages ? DEV_BAD_CACHE : 0;
  }
  __syncthreads();
}

// Hands out pages: this pass's sequence threadIdx.x takes need[threadIdx.x]
// pages behind its n_pages, `taken` pages after the first one handed out by
// this call. Warps take sequences, lanes their pages.
__device__ void take_pages(const ivc_cache& c, PlanShared& sh, const int32_t* seqs, int base, int n,
                           int free_count) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = warp; e < CA_THREADS && base + e < n; e += CA_WARPS) {
    const int need = sh.need[e];
    if (need == 0) continue;
    const int s = seq_of(seqs, base + e);
    const int have = c.n_pages[s];
    int32_t* row = c.table + static_cast<size_t>(s) * c.max_pages + have;
    for (int j = lane; j < need; j += 32) {
      const int at = free_count - 1 - (sh.order[e] + j);
      const int p = c.free_list[at];
      c.free_list[at] = -1;
      row[j] = p;
      if (page_ok(c, p)) c.ref[p] = 1;
      else atomicOr(&sh.bad, DEV_BAD_CACHE);
    }
    __syncwarp();
    if (lane == 0) c.n_pages[s] = have + need;
  }
}

// One holder less of page p; its bit is set when that was the last one.
__device__ void drop_page(const ivc_cache& c, PlanShared& sh, unsigned* freed, int p) {
  if (!page_ok(c, p)) {
    atomicOr(&sh.bad, DEV_BAD_CACHE);
    return;
  }
  const int before = atomicSub(&c.ref[p], 1);
  if (before == 1) {
    atomicOr(&freed[p >> 5], 1u << (p & 31));
  } else if (before < 1) {  // it belonged to nobody
    atomicAdd(&c.ref[p], 1);
    atomicOr(&sh.bad, DEV_BAD_CACHE);
  }
}

// Puts the pages of the bitmap on the free list, the lowest number on top.
__device__ void push_freed(const ivc_cache& c, PlanShared& sh, const unsigned* freed) {
  const int words = (c.pages + 31) / 32;
  long long mine = 0, total;
  for (int i = threadIdx.x; i < words; i += CA_THREADS) mine += __popc(freed[i]);
  block_scan(mine, sh.warp_sum, total);
  if (total == 0) return;
  const int fc = *c.free_count;
  long long carry = 0;
  for (int base = 0; base < words; base += CA_THREADS) {
    unsigned w = base + threadIdx.x < words ? freed[base + threadIdx.x] : 0u;
    long long sum;
    long long rank = carry + block_scan(__popc(w), sh.warp_sum, sum);
    while (w) {
      const int b = __ffs(w) - 1;
      w &= w - 1;
      const long long at = fc + total - 1 - rank++;
      if (at < c.pages) c.free_list[at] = (base + threadIdx.x) * 32 + b;
      else atomicOr(&sh.bad, DEV_BAD_CACHE);
    }
    carry += sum;
  }
  __syncthreads();
  if (threadIdx.x == 0) *c.free_count = static_cast<int>(min(fc + total, (long long)c.pages));
}

__device__ void clear_freed(const ivc_cache& c, unsigned* freed) {
  for (int i = threadIdx.x; i < (c.pages + 31) / 32; i += CA_THREADS) freed[i] = 0;
}

__global__ void __launch_bounds__(256) cache_init_kernel(ivc_cache c) {
  pdl_wait();
  pdl_trigger();
  const size_t cells = static_cast<size_t>(c.max_seqs) * c.max_pages;
  const size_t step = static_cast<size_t>(gridDim.x) * blockDim.x;
  const size_t t = static_cast<size_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  for (size_t i = t; i < cells; i += step) c.table[i] = -1;
  for (size_t i = t; i < static_cast<size_t>(c.max_seqs); i += step) c.length[i] = c.n_pages[i] = 0;
  for (size_t i = t; i < static_cast<size_t>(c.pages); i += step) {
    c.ref[i] = 0;
    c.free_list[i] = c.pages - 1 - static_cast<int>(i);
  }
  if (t == 0) *c.free_count = c.pages;
}

__global__ void __launch_bounds__(CA_THREADS)
    cache_reserve_kernel(ivc_cache c, const int32_t* tokens, const int32_t* seqs, int n,
                         int* status) {
  __shared__ PlanShared sh;
  pdl_wait();
  pdl_trigger();
  plan_begin(c, sh);
  const int fc = *c.free_count;
  // pages a sequence lacks for length + tokens[i] tokens
  auto lacks = [&](int i, int s, int& bad) -> int {
    if (tokens[i] < 0) { bad = DEV_BAD_CACHE; return 0; }
    const long long want = (static_cast<long long>(c.length[s]) + tokens[i] + c.page_tokens - 1) /
                           c.page_tokens;
    if (want > c.max_pages) { bad = DEV_CACHE_FULL; return 0; }
    return want > c.n_pages[s] ? static_cast<int>(want) - c.n_pages[s] : 0;
  };
  long long need = 0, total;
  for (int i = threadIdx.x; i < n; i += CA_THREADS) {
    const int s = seq_of(seqs, i);
    int bad = claim_seq(c, sh, s);
    if (!bad) bad = seq_sound(c, s);
    if (!bad) need += lacks(i, s, bad);
    if (bad) atomicOr(&sh.bad, bad);
  }
  block_scan(need, sh.warp_sum, total);
  if (threadIdx.x == 0 && total > fc) sh.bad |= DEV_CACHE_FULL;
  __syncthreads();
  if (sh.bad == 0 && total > 0) {
    long long carry = 0;
    for (int base = 0; base < n; base += CA_THREADS) {
      const int i = base + threadIdx.x;
      int ignored = 0;
      const int mine = i < n ? lacks(i, seq_of(seqs, i), ignored) : 0;
      long long sum;
      sh.order[threadIdx.x] = static_cast<int>(carry + block_scan(mine, sh.warp_sum, sum));
      sh.need[threadIdx.x] = mine;
      __syncthreads();
      take_pages(c, sh, seqs, base, n, fc);
      carry += sum;
      __syncthreads();
    }
    if (threadIdx.x == 0) *c.free_count = fc - static_cast<int>(total);
  }
  __syncthreads();
  if (threadIdx.x == 0 && sh.bad) atomicOr(status, sh.bad);
}

__global__ void __launch_bounds__(CA_THREADS)
    cache_free_kernel(ivc_cache c, const int32_t* seqs, int n, int* status) {
  extern __shared__ unsigned freed[];
  __shared__ PlanShared sh;
  pdl_wait();
  pdl_trigger();
  plan_begin(c, sh);
  clear_freed(c, freed);
  for (int i = threadIdx.x; i < n; i += CA_THREADS) {
    const int s = seq_of(seqs, i);
    int bad = claim_seq(c, sh, s);
    if (!bad) bad = seq_sound(c, s);
    if (bad) atomicOr(&sh.bad, bad);
  }
  __syncthreads();
  if (sh.bad == 0) {
    __syncthreads();  // drop_page may set bad: nobody decides by it any more
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = warp; i < n; i += CA_WARPS) {
      const int s = seq_of(seqs, i);
      const int np = c.n_pages[s];
      int32_t* row = c.table + static_cast<size_t>(s) * c.max_pages;
      for (int j = lane; j < np; j += 32) {
        drop_page(c, sh, freed, row[j]);
        row[j] = -1;
      }
      __syncwarp();
      if (lane == 0) c.n_pages[s] = c.length[s] = 0;
    }
    __syncthreads();
    push_freed(c, sh, freed);
  }
  __syncthreads();
  if (threadIdx.x == 0 && sh.bad) atomicOr(status, sh.bad);
}

// Workspace of fork and compact, after the 256-byte header.
struct ForkPlan {
  int32_t* n_jobs;    // [1]
  int32_t* len;       // [n] source lengths as they stood before the call
  int4* jobs;         // one per page copied (at most every page): {source, new page, rows, 0}
};
struct CompactPlan {
  int32_t* count;     // [n] tokens to move, 0 when the call is refused
  int2* rows;         // [n, keep_stride]: {source, target} token slot (page * page_tokens + slot)
};

__global__ void __launch_bounds__(CA_THREADS)
    cache_fork_kernel(ivc_cache c, const int32_t* src, const int32_t* dst, int n, int share,
                      ForkPlan plan, int* status) {
  __shared__ PlanShared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  plan_begin(c, sh);
  const int fc = *c.free_count;
  const int pt = c.page_tokens;
  auto copied = [&](int len) { return share ? (len % pt != 0) : (len + pt - 1) / pt; };
  long long need = 0, total;
  for (int i = threadIdx.x; i < n; i += CA_THREADS) {
    const int s = src[i], d = dst[i];
    int bad = claim_seq(c, sh, d);
    if (!bad && (s < 0 || s >= c.max_seqs)) bad = DEV_BAD_CACHE;
    if (!bad) bad = seq_sound(c, s);
    if (!bad && (c.n_pages[d] != 0 || c.length[d] != 0)) bad = DEV_BAD_CACHE;
    if (bad) {
      atomicOr(&sh.bad, bad);
      continue;
    }
    const int len = c.length[s];
    plan.len[i] = len;
    need += copied(len);
  }
  block_scan(need, sh.warp_sum, total);
  if (threadIdx.x == 0 && total > fc) sh.bad |= DEV_CACHE_FULL;
  __syncthreads();
  bool go = sh.bad == 0;
  __syncthreads();
  if (go) {  // the pages that are read or shared have to be pages
    for (int i = warp; i < n; i += CA_WARPS) {
      const int32_t* row = c.table + static_cast<size_t>(src[i]) * c.max_pages;
      for (int j = lane; j < (plan.len[i] + pt - 1) / pt; j += 32)
        if (!page_ok(c, row[j]) || c.ref[row[j]] < 1) atomicOr(&sh.bad, DEV_BAD_CACHE);
    }
    __syncthreads();
    go = sh.bad == 0;
    __syncthreads();
  }
  if (go) {
    // the shared pages first: a new sequence's own pages come behind them
    for (int i = warp; i < n; i += CA_WARPS) {
      const int full = share ? plan.len[i] / pt : 0;
      const int32_t* from = c.table + static_cast<size_t>(src[i]) * c.max_pages;
      int32_t* to = c.table + static_cast<size_t>(dst[i]) * c.max_pages;
      for (int j = lane; j < full; j += 32) {
        to[j] = from[j];
        atomicAdd(&c.ref[from[j]], 1);
      }
      if (lane == 0) {
        c.n_pages[dst[i]] = full;
        c.length[dst[i]] = plan.len[i];
      }
    }
    __syncthreads();
    long long carry = 0;
    for (int base = 0; base < n; base += CA_THREADS) {
      const int i = base + threadIdx.x;
      const int mine = i < n ? copied(plan.len[i]) : 0;
      long long sum;
      sh.order[threadIdx.x] = static_cast<int>(carry + block_scan(mine, sh.warp_sum, sum));
      sh.need[threadIdx.x] = mine;
      __syncthreads();
      take_pages(c, sh, dst, base, n, fc);
      __syncthreads();
      for (int e = warp; e < CA_THREADS && base + e < n; e += CA_WARPS) {
        const int len = plan.len[base + e], k = sh.need[e];
        const int first = (len + pt - 1) / pt - k;
        const int32_t* from = c.table + static_cast<size_t>(src[base + e]) * c.max_pages + first;
        const int32_t* to = c.table + static_cast<size_t>(dst[base + e]) * c.max_pages + first;
        for (int j = lane; j < k; j += 32)
          plan.jobs[sh.order[e] + j] =
              make_int4(from[j], to[j], min(pt, len - (first + j) * pt), 0);
      }
      carry += sum;
      __syncthreads();
    }
    if (threadIdx.x == 0) *c.free_count = fc - static_cast<int>(total);
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    *plan.n_jobs = go ? static_cast<int>(total) : 0;
    if (sh.bad) atomicOr(status, sh.bad);
  }
}

// Copies the jobs' rows in every layer, head, and of keys and values: one
// (job, plane, head) is rows * head_dim contiguous values, taken in chunks of 4 KB,
// a warp each with all of its loads in flight. (A CTA per (job, plane, head) left
// three quarters of its threads idle for 16-token pages.) Bound by HBM: three
// prefixes of up to 3390 tokens in 36 layers, 2.9 GB read and written, take 490 us.
constexpr int CC_PIECES = 8;  // 16-byte pieces per lane and chunk
__global__ void __launch_bounds__(256, 4) cache_copy_kernel(ivc_cache c, ForkPlan plan) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const unsigned per_row = c.head_dim / 8;  // 16-byte pieces
  const unsigned heads = c.kv_heads, planes = 2 * c.layers;
  const unsigned block = c.page_tokens * per_row;                       // a page of one head
  const unsigned chunks = (block + 32 * CC_PIECES - 1) / (32 * CC_PIECES);
  const unsigned long long units =
      static_cast<unsigned long long>(*plan.n_jobs) * planes * heads * chunks;
  const unsigned long long step = static_cast<unsigned long long>(gridDim.x) * (blockDim.x / 32);
  for (unsigned long long u = static_cast<unsigned long long>(blockIdx.x) * (blockDim.x / 32) +
                              (threadIdx.x >> 5);
       u < units; u += step) {
    // chunk fastest, then head, plane, job
    const unsigned per_job = planes * heads * chunks;                  // < 2^32: see cache_ok
    const unsigned job_no = static_cast<unsigned>(u / per_job);
    unsigned rest = static_cast<unsigned>(u - static_cast<unsigned long long>(job_no) * per_job);
    const unsigned chunk = rest % chunks;
    rest /= chunks;
    const unsigned h = rest % heads, plane = rest / heads;
    const int4 job = plan.jobs[job_no];
    const unsigned pieces = job.z * per_row, first = chunk * 32 * CC_PIECES + lane;
    if (chunk * 32 * CC_PIECES >= pieces || !page_ok(c, job.x) || !page_ok(c, job.y)) continue;
    uint4* base = static_cast<uint4*>(plane & 1 ? c.v : c.k);
    const size_t layer = static_cast<size_t>(plane >> 1) * c.pages;
    const uint4* from = base + ((layer + job.x) * heads + h) * block;
    uint4* to = base + ((layer + job.y) * heads + h) * block;
    uint4 r[CC_PIECES];
#pragma unroll
    for (int k = 0; k < CC_PIECES; ++k)
      if (first + 32 * k < pieces) r[k] = from[first + 32 * k];
#pragma unroll
    for (int k = 0; k < CC_PIECES; ++k)
      if (first + 32 * k < pieces) to[first + 32 * k] = r[k];
  }
}

__global__ void __launch_bounds__(CA_THREADS)
    cache_compact_kernel(ivc_cache c, const int32_t* count, const int32_t* keep, int stride,
                         const int32_t* start, const int32_t* seqs, int n, CompactPlan plan,
                         int* status) {
  extern __shared__ unsigned freed[];
  __shared__ PlanShared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  plan_begin(c, sh);
  clear_freed(c, freed);
  const int pt = c.page_tokens;
  auto first_of = [&](int i, int s) { return start ? start[i] : c.length[s]; };
  for (int i = threadIdx.x; i < n; i += CA_THREADS) {
    const int s = seq_of(seqs, i);
    int bad = claim_seq(c, sh, s);
    if (!bad) bad = seq_sound(c, s);
    if (!bad) {
      const long long a = first_of(i, s), m = count[i];
      if (a < 0 || a > c.length[s] || m < 0 || (keep && m > stride) ||
          a + m > static_cast<long long>(c.n_pages[s]) * pt) {
        bad = DEV_BAD_CACHE;
      } else if ((a + m) % pt != 0) {  // the partly filled last page is nobody else's
        const int p = c.table[static_cast<size_t>(s) * c.max_pages + (a + m) / pt];
        if (!page_ok(c, p) || c.ref[p] != 1) bad = DEV_BAD_CACHE;
      }
    }
    if (bad) atomicOr(&sh.bad, bad);
  }
  __syncthreads();
  bool go = sh.bad == 0;
  __syncthreads();
  if (go && keep) {
    // every kept token on its own: rising, held, and its target a page of this
    // sequence alone
    const long long cells = static_cast<long long>(n) * stride;
    for (long long e = threadIdx.x; e < cells; e += CA_THREADS) {
      const int i = static_cast<int>(e / stride), j = static_cast<int>(e % stride);
      if (j >= count[i]) continue;
      const int s = seq_of(seqs, i);
      const int32_t* row = c.table + static_cast<size_t>(s) * c.max_pages;
      const long long a = first_of(i, s), k = keep[e];
      const long long from = a + k, to = a + j;
      const bool rises = k >= 0 && (j == 0 || keep[e - 1] < k);
      if (!rises || from < to || from >= static_cast<long long>(c.n_pages[s]) * pt) {
        atomicOr(&sh.bad, DEV_BAD_CACHE);
        continue;
      }
      const int pf = row[from / pt], pd = row[to / pt];
      if (!page_ok(c, pf) || !page_ok(c, pd) || (from != to && c.ref[pd] != 1)) {
        atomicOr(&sh.bad, DEV_BAD_CACHE);
        continue;
      }
      plan.rows[e] = make_int2(pf * pt + static_cast<int>(from % pt),
                               pd * pt + static_cast<int>(to % pt));
    }
    __syncthreads();
    go = sh.bad == 0;
    __syncthreads();
  }
  if (keep)
    for (int i = threadIdx.x; i < n; i += CA_THREADS) plan.count[i] = go ? count[i] : 0;
  if (go) {
    for (int i = warp; i < n; i += CA_WARPS) {
      const int s = seq_of(seqs, i);
      const int len = first_of(i, s) + count[i];
      const int np = c.n_pages[s], left = (len + pt - 1) / pt;
      int32_t* row = c.table + static_cast<size_t>(s) * c.max_pages;
      for (int j = left + lane; j < np; j += 32) {
        drop_page(c, sh, freed, row[j]);
        row[j] = -1;
      }
      __syncwarp();
      if (lane == 0) {
        c.length[s] = len;
        c.n_pages[s] = min(np, left);
      }
    }
    __syncthreads();
    push_freed(c, sh, freed);
  }
  __syncthreads();
  if (threadIdx.x == 0 && sh.bad) atomicOr(status, sh.bad);
}

// Moves the kept tokens of one sequence, plane (layer, keys or values) and
// group of heads, in place. Targets do not lie behind their sources and rise
// with them, so a chunk of rows that is read whole before any of it is written
// cannot spoil a later chunk's sources; the next chunk's loads are issued before
// this one's stores (its sources lie behind these targets). Bound by HBM: 848 of 3390
// tokens of three sequences in 36 layers, 0.7 GB read and written, take 145 us.
constexpr int MV_THREADS = 256;
constexpr int MV_PIECES = 4;  // 16-byte pieces a thread holds of a chunk
constexpr int MV_CTAS = 8;
__global__ void __launch_bounds__(MV_THREADS, 4)
    cache_move_kernel(ivc_cache c, CompactPlan plan, int stride, int head_groups,
                      int heads_per_group) {
  pdl_wait();
  pdl_trigger();
  const int i = blockIdx.x / head_groups;
  const unsigned h0 = (blockIdx.x % head_groups) * heads_per_group;
  const unsigned heads = min(heads_per_group, c.kv_heads - static_cast<int>(h0));
  const int plane = blockIdx.y;
  const int n = plan.count[i];
  if (n == 0) return;
  const int row_log = c.head_dim == 64 ? 3 : 4;          // 16-byte pieces of a row
  const int pt_log = 31 - __clz(c.page_tokens);
  const int2* rows = plan.rows + static_cast<size_t>(i) * stride;
  uint4* base = static_cast<uint4*>(plane & 1 ? c.v : c.k) +
                ((static_cast<size_t>(plane >> 1) * c.pages * c.kv_heads) << (pt_log + row_log));
  // piece x of the group: 16 bytes of head x / 2^row_log % heads of kept token
  // x / 2^row_log / heads
  const unsigned pieces = (static_cast<unsigned>(n) * heads) << row_log;  // < 2^31: see below
  auto at = [&](int slot, unsigned h, unsigned piece) {
    const size_t page = slot >> pt_log;
    return ((((page * c.kv_heads + h0 + h) << pt_log) + (slot & (c.page_tokens - 1))) << row_log) + piece;
  };
  struct Chunk {
    uint4 r[MV_PIECES];
    int slot[MV_PIECES];  // the target, -1: nothing to move
  };
  auto split = [&](unsigned x, unsigned& h, unsigned& piece) {
    piece = x & ((1u << row_log) - 1);
    const unsigned token = (x >> row_log) / heads;
    h = (x >> row_log) - token * heads;
    return token;
  };
  auto load = [&](Chunk& k, unsigned x0) {
#pragma unroll
    for (int e = 0; e < MV_PIECES; ++e) {
      const unsigned x = x0 + e * MV_THREADS + threadIdx.x;
      k.slot[e] = -1;
      if (x < pieces) {
        unsigned h, piece;
        const int2 row = rows[split(x, h, piece)];
        if (row.x != row.y) {
          k.slot[e] = row.y;
          k.r[e] = base[at(row.x, h, piece)];
        }
      }
    }
  };
  Chunk now, next;
  load(now, 0);
  for (unsigned x0 = 0; x0 < pieces; x0 += MV_PIECES * MV_THREADS) {
    const bool more = x0 + MV_PIECES * MV_THREADS < pieces;
    if (more) load(next, x0 + MV_PIECES * MV_THREADS);
    __syncthreads();  // the chunk is read
#pragma unroll
    for (int e = 0; e < MV_PIECES; ++e)
      if (now.slot[e] >= 0) {
        unsigned h, piece;
        split(x0 + e * MV_THREADS + threadIdx.x, h, piece);
        base[at(now.slot[e], h, piece)] = now.r[e];
      }
    if (more) now = next;
  }
}

size_t up256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

size_t fork_ws(const ivc_cache* c, int n) {
  const size_t want = static_cast<size_t>(n) * c->max_pages, most = c->pages;
  return 256 + 256 + up256(static_cast<size_t>(n) * 4) +
         (want < most ? want : most) * sizeof(int4);
}
size_t compact_ws(int n, int stride) {
  return 256 + up256(static_cast<size_t>(n) * 4) + static_cast<size_t>(n) * stride * sizeof(int2);
}

size_t bitmap_bytes(const ivc_cache* c) { return static_cast<size_t>((c->pages + 31) / 32) * 4; }

}  // namespace

int step_ws_ok(const void* ws, size_t have, size_t need) {
  if (!ws) return IVC_EINVAL;
  if (reinterpret_cast<uintptr_t>(ws) & 255u) return IVC_EALIGN;
  return have < need ? IVC_EWORKSPACE : IVC_OK;
}

int cache_ok(const ivc_cache* c) {
  if (!c || c->layers < 1 || c->pages < 1 || c->kv_heads < 1 || c->max_seqs < 1 || c->max_pages < 1)
    return IVC_EINVAL;
  if (!c->k || !c->v || !c->table || !c->length || !c->n_pages || !c->ref || !c->free_list ||
      !c->free_count)
    return IVC_EINVAL;
  const int pt = c->page_tokens;
  if (pt != 16 && pt != 32 && pt != 64 && pt != 128) return IVC_EUNSUPPORTED;
  if (c->head_dim != 64 && c->head_dim != 128) return IVC_EUNSUPPORTED;
  if (c->pages > CA_MAX_PAGES || c->max_seqs > CA_MAX_SEQS || c->kv_heads > 1024 ||
      c->layers > 4096)
    return IVC_EUNSUPPORTED;
  if (static_cast<long long>(c->max_pages) * pt > (1ll << 30)) return IVC_EUNSUPPORTED;
  if (static_cast<long long>(c->pages) * c->kv_heads * pt >= (1ll << 31)) return IVC_EUNSUPPORTED;
  auto off = [](const void* p, unsigned m) { return (reinterpret_cast<uintptr_t>(p) & m) != 0; };
  if (off(c->k, 15) || off(c->v, 15)) return IVC_EALIGN;
  for (const int32_t* p : {c->table, c->length, c->n_pages, c->ref, c->free_list, c->free_count})
    if (off(p, 3)) return IVC_EALIGN;
  return IVC_OK;
}

}  // namespace ivc

using namespace ivc;

extern "C" {

int ivc_cache_init(const ivc_cache* c, ivc_stream_t stream) {
  if (const int rc = cache_ok(c)) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  TraceScope ts("cache.init", s);
  return launch_k(cache_init_kernel, dim3(num_sms()), dim3(256), 0, s, 1, *c);
}

size_t ivc_cache_workspace_size(const ivc_cache* c, int n, int keep_stride) {
  if (cache_ok(c) != IVC_OK || n < 0 || n > c->max_seqs || keep_stride < 0) return 0;
  const size_t a = fork_ws(c, n), b = compact_ws(n, keep_stride);
  return a > b ? a : b;
}

int ivc_cache_reserve(const ivc_cache* c, const int32_t* tokens, const int32_t* seqs, int n,
                      void* workspace, size_t ws_bytes, ivc_stream_t stream) {
  if (const int rc = cache_ok(c)) return rc;
  if (n < 0 || n > c->max_seqs || (n > 0 && !tokens)) return IVC_EINVAL;
  if (const int rc = step_ws_ok(workspace, ws_bytes, IVC_STEP_WORKSPACE_BYTES)) return rc;
  if (n == 0) return IVC_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  TraceScope ts("cache.reserve", s);
  return launch_k(cache_reserve_kernel, dim3(1), dim3(CA_THREADS), 0, s, 1, *c, tokens, seqs, n,
                  static_cast<int*>(workspace));
}

int ivc_cache_free(const ivc_cache* c, const int32_t* seqs, int n, void* workspace,
                   size_t ws_bytes, ivc_stream_t stream) {
  if (const int rc = cache_ok(c)) return rc;
  if (n < 0 || n > c->max_seqs) return IVC_EINVAL;
  if (const int rc = step_ws_ok(workspace, ws_bytes, IVC_STEP_WORKSPACE_BYTES)) return rc;
  if (n == 0) return IVC_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const size_t smem = bitmap_bytes(c);
  if (const int rc = smem_optin(reinterpret_cast<const void*>(cache_free_kernel), smem)) return rc;
  TraceScope ts("cache.free", s);
  return launch_k(cache_free_kernel, dim3(1), dim3(CA_THREADS), smem, s, 1, *c, seqs, n,
                  static_cast<int*>(workspace));
}

int ivc_cache_fork(const ivc_cache* c, const int32_t* src, const int32_t* dst, int n, int share,
                   void* workspace, size_t ws_bytes, ivc_stream_t stream) {
  if (const int rc = cache_ok(c)) return rc;
  if (n < 0 || n > c->max_seqs || (n > 0 && (!src || !dst))) return IVC_EINVAL;
  if (const int rc = step_ws_ok(workspace, ws_bytes, fork_ws(c, n))) return rc;
  if (n == 0) return IVC_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* w = static_cast<char*>(workspace) + 256;
  ForkPlan plan;
  plan.n_jobs = reinterpret_cast<int32_t*>(w);
  plan.len = reinterpret_cast<int32_t*>(w + 256);
  plan.jobs = reinterpret_cast<int4*>(w + 256 + up256(static_cast<size_t>(n) * 4));
  {
    TraceScope ts("cache.fork", s);
    const int rc = launch_k(cache_fork_kernel, dim3(1), dim3(CA_THREADS), 0, s, 1, *c, src, dst, n,
                            share, plan, static_cast<int*>(workspace));
    if (rc != IVC_OK) return rc;
  }
  TraceScope ts("cache.copy", s);
  return launch_k(cache_copy_kernel, dim3(4 * num_sms()), dim3(256), 0, s, 1, *c, plan);
}

int ivc_cache_compact(const ivc_cache* c, const int32_t* count, const int32_t* keep,
                      int keep_stride, const int32_t* start, const int32_t* seqs, int n,
                      void* workspace, size_t ws_bytes, ivc_stream_t stream) {
  if (const int rc = cache_ok(c)) return rc;
  if (n < 0 || n > c->max_seqs || keep_stride < 0 || (n > 0 && !count)) return IVC_EINVAL;
  const int stride = keep ? keep_stride : 0;
  if (const int rc = step_ws_ok(workspace, ws_bytes, compact_ws(n, stride))) return rc;
  if (n == 0) return IVC_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* w = static_cast<char*>(workspace) + 256;
  CompactPlan plan;
  plan.count = reinterpret_cast<int32_t*>(w);
  plan.rows = reinterpret_cast<int2*>(w + up256(static_cast<size_t>(n) * 4));
  const size_t smem = bitmap_bytes(c);
  if (const int rc = smem_optin(reinterpret_cast<const void*>(cache_compact_kernel), smem)) return rc;
  {
    TraceScope ts("cache.compact", s);
    const int rc = launch_k(cache_compact_kernel, dim3(1), dim3(CA_THREADS), smem, s, 1, *c, count,
                            keep, stride, start, seqs, n, plan, static_cast<int*>(workspace));
    if (rc != IVC_OK) return rc;
  }
  if (stride == 0) return IVC_OK;
  // A CTA takes as many heads as leaves MV_CTAS CTAs per SM. (Not by the keep
  // lists' width, which says little of the counts: for 48 paths of 7 tokens in lists
  // 128 wide, reserve and compact took 79 us with a CTA per head and take 42.) 4 per
  // SM: 697 against 670 us for the thinned prefixes; 16: the same. A sequence's tokens are at most
  // pages * page_tokens <= 2^27, and a head 16 pieces; more heads than one only
  // where that stays in 32 bits.
  const long long planes = 2ll * n * c->layers, wanted = MV_CTAS * num_sms();
  int per_group = static_cast<int>(c->kv_heads * planes / wanted);
  const long long most = (1ll << 31) / 16 / (static_cast<long long>(c->pages) * c->page_tokens);
  if (per_group > most) per_group = static_cast<int>(most);
  per_group = per_group < 1 ? 1 : per_group > c->kv_heads ? c->kv_heads : per_group;
  const int groups = (c->kv_heads + per_group - 1) / per_group;
  TraceScope ts("cache.move", s);
  return launch_k(cache_move_kernel, dim3(static_cast<unsigned>(n) * groups, 2 * c->layers),
                  dim3(MV_THREADS), 0, s, 1, *c, plan, stride, groups, per_group);
}

}  // extern "C"
