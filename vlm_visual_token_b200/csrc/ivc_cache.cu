// ivc_cache.cu — pages of the key/value cache behind the spliced sequence:
// taking, sharing, copying, compacting and giving them back.
//
// Each operation is a device plan and (fork, compact) a move of rows by that
// plan, as in the sequence assembly (ivc_assemble.cu): no length or page number
// is read on the host, so a call can be captured and replayed.
//
// The plan is one CTA. It first checks everything that the operation is going
// to touch, and only when all of it is sound changes the tables: a refused call
// leaves the cache as it was. (Holders of pages to be given back are counted down
// to see that there are enough of them, and up again where there are not.) Counts
// are integers and pages are handed out by prefix sums, so results do not depend on
// thread order; freed pages are collected as bits of a bitmap in shared memory (one
// bit per page, at most 128 KB), which both finds the last holder's release exactly
// once and lists the freed pages in ascending order.
#include <cuda_runtime.h>

#include "ivc_internal.h"
#include "ivc_ptx.cuh"

namespace ivc {
namespace {

constexpr int CA_THREADS = 1024;
constexpr int CA_WARPS = CA_THREADS / 32;
constexpr int CA_MAX_SEQS = 65536;
constexpr int CA_MAX_PAGES = 1 << 20;

// What the plan kernels keep in shared memory besides the page bitmap. The
// sequences of a call are taken in passes of CA_THREADS, a thread each; their pages
// by all threads (see pages_of_pass).
struct PlanShared {
  unsigned seen[CA_MAX_SEQS / 32];  // sequences named by this call
  int seq[CA_THREADS];              // of this pass
  int from[CA_THREADS];             // fork: the source; compact: the first token
  int len[CA_THREADS];              // committed tokens; compact: tokens kept
  int np[CA_THREADS];               // pages held
  int order[CA_THREADS];            // pages taken before this sequence's
  int need[CA_THREADS];             // pages it takes
  long long warp_sum[CA_WARPS];
  int widest;                       // compact: the most tokens kept of one sequence
  int bad;                          // DEV_* bits
};

// Calls f(e, j) for every page j < count(e) of every sequence e < m of a pass: as
// many neighbouring threads per sequence as there are, so that a few sequences'
// pages and many sequences' are read in few dependent steps.
template <typename Count, typename F>
__device__ __forceinline__ void pages_of_pass(int m, Count count, F f) {
  const int lanes = 1 << (31 - __clz(CA_THREADS / max(m, 1)));  // m * lanes <= CA_THREADS
  const int e = threadIdx.x / lanes;
  if (e >= m) return;
  const int n = count(e);
  for (int j = threadIdx.x % lanes; j < n; j += lanes) f(e, j);
}

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

// The pages on the free list, once `seen` is clear.
__device__ int plan_begin(const ivc_cache& c, PlanShared& sh) {
  const int fc = *c.free_count;
  for (int i = threadIdx.x; i < (c.max_seqs + 31) / 32; i += CA_THREADS) sh.seen[i] = 0;
  if (threadIdx.x == 0) sh.bad = fc < 0 || fc > c.pages ? DEV_BAD_CACHE : 0;
  __syncthreads();
  return fc;
}

// Whether everything was sound so far: the same in every thread, and nobody sets
// sh.bad before all have read it.
__device__ bool still_good(const PlanShared& sh) {
  __syncthreads();
  const bool good = sh.bad == 0;
  __syncthreads();
  return good;
}

// Clears the bitmap of pages; a barrier of the plan stands before its first use.
__device__ void clear_pages(const ivc_cache& c, unsigned* pages) {
  for (int i = threadIdx.x; i < (c.pages + 31) / 32; i += CA_THREADS) pages[i] = 0;
}

// The `total` pages on top of the free list are pages that nobody holds, each there
// once (a bit per page in `taken`, which is clear). Without this a page listed twice or
// still held would get two owners, and the next store would spoil another sequence.
__device__ void check_top(const ivc_cache& c, PlanShared& sh, unsigned* taken, int free_count,
                          int total) {
  for (int k = threadIdx.x; k < total; k += CA_THREADS) {
    const int p = c.free_list[free_count - 1 - k];
    const unsigned bit = 1u << (p & 31);
    if (!page_ok(c, p) || c.ref[p] != 0 || (atomicOr(&taken[p >> 5], bit) & bit))
      atomicOr(&sh.bad, DEV_BAD_CACHE);
  }
}

// The k-th page that this call takes off the free list.
__device__ __forceinline__ int take_page(const ivc_cache& c, int free_count, int k) {
  const int at = free_count - 1 - k;
  const int p = c.free_list[at];
  c.free_list[at] = -1;
  c.ref[p] = 1;
  return p;
}

// One holder less of page p; its bit is set when that was the last one. A page that is
// none or belongs to nobody makes the call bad, and give_back then takes all back.
__device__ void drop_page(const ivc_cache& c, PlanShared& sh, unsigned* freed, int p) {
  if (!page_ok(c, p)) {
    atomicOr(&sh.bad, DEV_BAD_CACHE);
    return;
  }
  const int before = atomicSub(&c.ref[p], 1);
  if (before == 1) atomicOr(&freed[p >> 5], 1u << (p & 31));
  else if (before < 1) atomicOr(&sh.bad, DEV_BAD_CACHE);
}

// Puts the `total` pages of the bitmap behind the `fc` on the free list, the lowest
// number on top; there is room for them.
__device__ void push_freed(const ivc_cache& c, PlanShared& sh, const unsigned* freed, int fc,
                           long long total) {
  const int words = (c.pages + 31) / 32;
  long long carry = 0;
  for (int base = 0; base < words; base += CA_THREADS) {
    unsigned w = base + threadIdx.x < words ? freed[base + threadIdx.x] : 0u;
    long long sum;
    long long rank = carry + block_scan(__popc(w), sh.warp_sum, sum);
    while (w) {
      const int b = __ffs(w) - 1;
      w &= w - 1;
      c.free_list[fc + total - 1 - rank++] = (base + threadIdx.x) * 32 + b;
    }
    carry += sum;
  }
  if (threadIdx.x == 0) *c.free_count = fc + static_cast<int>(total);
}

// Gives back the pages that `each` names (it calls its argument with the address of
// every table entry concerned, all threads together), if all of them are pages with a
// holder and the list has room for those freed; else everything stays as it was. The
// holders are counted first, which finds a wrong entry behind right ones and a page
// named more often than it is held, and counted back where one was found.
template <typename Each>
__device__ bool give_back(const ivc_cache& c, PlanShared& sh, unsigned* freed, int fc, Each each) {
  each([&](int32_t* at) { drop_page(c, sh, freed, *at); });
  __syncthreads();  // the bitmap is complete
  long long mine = 0, total;
  for (int i = threadIdx.x; i < (c.pages + 31) / 32; i += CA_THREADS) mine += __popc(freed[i]);
  block_scan(mine, sh.warp_sum, total);
  if (threadIdx.x == 0 && fc + total > c.pages) sh.bad |= DEV_BAD_CACHE;
  if (!still_good(sh)) {
    each([&](int32_t* at) {
      if (page_ok(c, *at)) atomicAdd(&c.ref[*at], 1);
    });
    return false;
  }
  each([&](int32_t* at) { *at = -1; });
  if (total > 0) push_freed(c, sh, freed, fc, total);
  return true;
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
  extern __shared__ unsigned taken[];
  __shared__ PlanShared sh;
  pdl_wait();
  pdl_trigger();
  const int fc = plan_begin(c, sh);
  clear_pages(c, taken);
  const int tid = threadIdx.x;
  // sequence base + tid: its number, pages, and the pages it lacks for length +
  // tokens[] tokens, into shared memory
  auto read = [&](int base, bool first_time) {
    const int i = base + tid;
    int bad = 0, s = 0, need = 0;
    if (i < n) {
      s = seq_of(seqs, i);
      if (first_time) bad = claim_seq(c, sh, s);
      if (!bad) bad = seq_sound(c, s);
      if (!bad) {
        const int np = c.n_pages[s];
        const long long want =
            (static_cast<long long>(c.length[s]) + tokens[i] + c.page_tokens - 1) / c.page_tokens;
        if (tokens[i] < 0) bad = DEV_BAD_CACHE;
        else if (want > c.max_pages) bad = DEV_CACHE_FULL;
        else if (want > np) need = static_cast<int>(want) - np;
        sh.np[tid] = np;
      }
      if (bad) atomicOr(&sh.bad, bad);
    }
    sh.seq[tid] = s;
    sh.need[tid] = need;
    return need;
  };
  long long need = 0, total;
  for (int base = 0; base < n; base += CA_THREADS) need += read(base, true);
  block_scan(need, sh.warp_sum, total);
  if (total > fc) {
    if (tid == 0) sh.bad |= DEV_CACHE_FULL;
  } else if (fc <= c.pages) {
    check_top(c, sh, taken, fc, static_cast<int>(total));
  }
  if (still_good(sh) && total > 0) {
    long long carry = 0;
    for (int base = 0; base < n; base += CA_THREADS) {
      if (n > CA_THREADS) read(base, false);
      const int m = min(CA_THREADS, n - base);
      long long sum;
      sh.order[tid] = static_cast<int>(carry + block_scan(sh.need[tid], sh.warp_sum, sum));
      __syncthreads();
      pages_of_pass(m, [&](int e) { return sh.need[e]; }, [&](int e, int j) {
        c.table[static_cast<size_t>(sh.seq[e]) * c.max_pages + sh.np[e] + j] =
            take_page(c, fc, sh.order[e] + j);
      });
      if (tid < m && sh.need[tid] > 0) c.n_pages[sh.seq[tid]] = sh.np[tid] + sh.need[tid];
      carry += sum;
      __syncthreads();
    }
    if (tid == 0) *c.free_count = fc - static_cast<int>(total);
  }
  __syncthreads();
  if (tid == 0 && sh.bad) atomicOr(status, sh.bad);
}

__global__ void __launch_bounds__(CA_THREADS)
    cache_free_kernel(ivc_cache c, const int32_t* seqs, int n, int* status) {
  extern __shared__ unsigned freed[];
  __shared__ PlanShared sh;
  pdl_wait();
  pdl_trigger();
  const int fc = plan_begin(c, sh);
  clear_pages(c, freed);
  const int tid = threadIdx.x;
  auto read = [&](int base, bool first_time) {
    const int i = base + tid;
    if (i >= n) return;
    const int s = seq_of(seqs, i);
    int bad = first_time ? claim_seq(c, sh, s) : 0;
    if (!bad) bad = seq_sound(c, s);
    if (bad) {
      atomicOr(&sh.bad, bad);
      return;
    }
    sh.seq[tid] = s;
    sh.np[tid] = c.n_pages[s];
  };
  // f(pass) with the sequences of each pass in shared memory
  auto passes = [&](auto f) {
    for (int base = 0; base < n; base += CA_THREADS) {
      if (n > CA_THREADS) {
        __syncthreads();
        read(base, false);
        __syncthreads();
      }
      f(min(CA_THREADS, n - base));
    }
  };
  for (int base = 0; base < n; base += CA_THREADS) read(base, true);
  if (still_good(sh) && give_back(c, sh, freed, fc, [&](auto f) {
        passes([&](int m) {
          pages_of_pass(m, [&](int e) { return sh.np[e]; }, [&](int e, int j) {
            f(c.table + static_cast<size_t>(sh.seq[e]) * c.max_pages + j);
          });
        });
      }))
    passes([&](int m) {
      if (tid < m) c.n_pages[sh.seq[tid]] = c.length[sh.seq[tid]] = 0;
    });
  __syncthreads();
  if (tid == 0 && sh.bad) atomicOr(status, sh.bad);
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
  extern __shared__ unsigned taken[];
  __shared__ PlanShared sh;
  pdl_wait();
  pdl_trigger();
  const int fc = plan_begin(c, sh);
  clear_pages(c, taken);
  const int tid = threadIdx.x, pt = c.page_tokens;
  auto copied = [&](int len) { return share ? (len % pt != 0) : (len + pt - 1) / pt; };
  auto table_of = [&](int s) { return c.table + static_cast<size_t>(s) * c.max_pages; };
  // pair base + tid into shared memory; later passes take the source's length as it
  // stood before the call (an earlier pass may have made the source a target)
  auto read = [&](int base, bool first_time) {
    const int i = base + tid;
    int bad = 0, need = 0;
    if (i < n) {
      const int s = src[i], d = dst[i];
      int len = 0;
      if (first_time) {
        bad = claim_seq(c, sh, d);
        if (!bad && (s < 0 || s >= c.max_seqs)) bad = DEV_BAD_CACHE;
        if (!bad) bad = seq_sound(c, s);
        if (!bad && (c.n_pages[d] != 0 || c.length[d] != 0)) bad = DEV_BAD_CACHE;
        if (!bad) len = plan.len[i] = c.length[s];
        if (bad) atomicOr(&sh.bad, bad);
      } else {
        len = plan.len[i];
      }
      need = bad ? 0 : copied(len);
      sh.seq[tid] = d;
      sh.from[tid] = s;
      sh.len[tid] = len;
    }
    sh.need[tid] = need;
    return need;
  };
  auto used = [&](int e) { return (sh.len[e] + pt - 1) / pt; };
  long long need = 0, total;
  for (int base = 0; base < n; base += CA_THREADS) need += read(base, true);
  block_scan(need, sh.warp_sum, total);
  if (tid == 0 && total > fc) sh.bad |= DEV_CACHE_FULL;
  bool go = still_good(sh);
  if (go) {  // the pages that are taken, read or shared have to be pages
    check_top(c, sh, taken, fc, static_cast<int>(total));
    for (int base = 0; base < n; base += CA_THREADS) {
      if (n > CA_THREADS) {
        __syncthreads();
        read(base, false);
        __syncthreads();
      }
      pages_of_pass(min(CA_THREADS, n - base), used, [&](int e, int j) {
        const int p = table_of(sh.from[e])[j];
        if (!page_ok(c, p) || c.ref[p] < 1) atomicOr(&sh.bad, DEV_BAD_CACHE);
      });
    }
    go = still_good(sh);
  }
  if (go) {
    long long carry = 0;
    for (int base = 0; base < n; base += CA_THREADS) {
      if (n > CA_THREADS) {
        __syncthreads();
        read(base, false);
      }
      const int m = min(CA_THREADS, n - base);
      long long sum;
      sh.order[tid] = static_cast<int>(carry + block_scan(sh.need[tid], sh.warp_sum, sum));
      __syncthreads();
      // the shared pages, and behind them new ones
      pages_of_pass(m, used, [&](int e, int j) {
        const int p = table_of(sh.from[e])[j], full = used(e) - sh.need[e];
        int mine = p;
        if (j < full) {
          atomicAdd(&c.ref[p], 1);
        } else {
          const int k = sh.order[e] + j - full;
          mine = take_page(c, fc, k);
          plan.jobs[k] = make_int4(p, mine, min(pt, sh.len[e] - j * pt), 0);
        }
        table_of(sh.seq[e])[j] = mine;
      });
      if (tid < m) {
        c.n_pages[sh.seq[tid]] = used(tid);
        c.length[sh.seq[tid]] = sh.len[tid];
      }
      carry += sum;
    }
    __syncthreads();
    if (tid == 0) *c.free_count = fc - static_cast<int>(total);
  }
  __syncthreads();
  if (tid == 0) {
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
  pdl_wait();
  pdl_trigger();
  const int fc = plan_begin(c, sh);
  clear_pages(c, freed);
  const int tid = threadIdx.x, pt = c.page_tokens;
  // sequence base + tid: its first token, kept tokens and pages, into shared memory
  auto read = [&](int base, bool first_time) {
    const int i = base + tid;
    if (i >= n) return;
    const int s = seq_of(seqs, i);
    int bad = first_time ? claim_seq(c, sh, s) : 0;
    if (!bad) bad = seq_sound(c, s);
    if (!bad) {
      const int len = c.length[s], np = c.n_pages[s];
      const long long a = start ? start[i] : len, m = count[i];
      if (a < 0 || a > len || m < 0 || (keep && m > stride) || a + m > static_cast<long long>(np) * pt) {
        bad = DEV_BAD_CACHE;
      } else if (first_time && (a + m) % pt != 0) {  // the partly filled last page is nobody else's
        const int p = c.table[static_cast<size_t>(s) * c.max_pages + (a + m) / pt];
        if (!page_ok(c, p) || c.ref[p] != 1) bad = DEV_BAD_CACHE;
      }
      sh.seq[tid] = s;
      sh.from[tid] = static_cast<int>(a);
      sh.len[tid] = static_cast<int>(m);
      sh.np[tid] = np;
    }
    if (bad) atomicOr(&sh.bad, bad);
  };
  for (int base = 0; base < n; base += CA_THREADS) read(base, true);
  bool go = still_good(sh);
  if (go && keep) {
    for (int base = 0; base < n; base += CA_THREADS) {
      if (n > CA_THREADS) {
        __syncthreads();
        read(base, false);
        __syncthreads();
      }
      // every kept token on its own: rising, held, and its target a page of this
      // sequence alone
      const int m = min(CA_THREADS, n - base);
      if (tid == 0) sh.widest = 0;
      __syncthreads();
      if (tid < m) atomicMax(&sh.widest, sh.len[tid]);
      __syncthreads();
      const int width = sh.widest;
      const long long cells = static_cast<long long>(m) * width;
      for (long long cell = tid; cell < cells; cell += CA_THREADS) {
        const int e = static_cast<int>(cell / width);
        const int j = static_cast<int>(cell - static_cast<long long>(e) * width);
        if (j >= sh.len[e]) continue;
        const size_t at = static_cast<size_t>(base + e) * stride + j;
        const int32_t* row = c.table + static_cast<size_t>(sh.seq[e]) * c.max_pages;
        const long long a = sh.from[e], k = keep[at];
        const long long from = a + k, to = a + j;
        const bool rises = k >= 0 && (j == 0 || keep[at - 1] < k);
        if (!rises || from < to || from >= static_cast<long long>(sh.np[e]) * pt) {
          atomicOr(&sh.bad, DEV_BAD_CACHE);
          continue;
        }
        const int pf = row[from / pt], pd = row[to / pt];
        if (!page_ok(c, pf) || !page_ok(c, pd) || (from != to && c.ref[pd] != 1)) {
          atomicOr(&sh.bad, DEV_BAD_CACHE);
          continue;
        }
        plan.rows[at] = make_int2(pf * pt + static_cast<int>(from % pt),
                                  pd * pt + static_cast<int>(to % pt));
      }
    }
    go = still_good(sh);
  }
  auto left = [&](int e) { return (sh.from[e] + sh.len[e] + pt - 1) / pt; };
  // f(pass) with the sequences of each pass in shared memory
  auto passes = [&](auto f) {
    for (int base = 0; base < n; base += CA_THREADS) {
      if (n > CA_THREADS) {
        __syncthreads();
        read(base, false);
        __syncthreads();
      }
      f(min(CA_THREADS, n - base));
    }
  };
  go = go && give_back(c, sh, freed, fc, [&](auto f) {
    passes([&](int m) {
      pages_of_pass(m, [&](int e) { return max(0, sh.np[e] - left(e)); }, [&](int e, int j) {
        f(c.table + static_cast<size_t>(sh.seq[e]) * c.max_pages + left(e) + j);
      });
    });
  });
  if (go)
    passes([&](int m) {
      if (tid < m) {
        c.length[sh.seq[tid]] = sh.from[tid] + sh.len[tid];
        c.n_pages[sh.seq[tid]] = min(sh.np[tid], left(tid));
      }
    });
  if (keep)
    for (int i = tid; i < n; i += CA_THREADS) plan.count[i] = go ? count[i] : 0;
  __syncthreads();
  if (tid == 0 && sh.bad) atomicOr(status, sh.bad);
}

// Moves the kept tokens of one sequence, plane (layer, keys or values) and
// group of heads, in place. Targets do not lie behind their sources and rise
// with them, so a chunk of rows that is read whole before any of it is written
// cannot spoil a later chunk's sources; the next chunk's loads are issued before
// this one's stores (its sources lie behind these targets). Bound by HBM: 848 of 3390
// tokens of three sequences in 36 layers, 0.7 GB read and written, take 149 us.
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
  const size_t smem = bitmap_bytes(c);
  if (const int rc = smem_optin(reinterpret_cast<const void*>(cache_reserve_kernel), smem)) return rc;
  TraceScope ts("cache.reserve", s);
  return launch_k(cache_reserve_kernel, dim3(1), dim3(CA_THREADS), smem, s, 1, *c, tokens, seqs, n,
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
  const size_t smem = bitmap_bytes(c);
  if (const int rc = smem_optin(reinterpret_cast<const void*>(cache_fork_kernel), smem)) return rc;
  {
    TraceScope ts("cache.fork", s);
    const int rc = launch_k(cache_fork_kernel, dim3(1), dim3(CA_THREADS), smem, s, 1, *c, src, dst, n,
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
