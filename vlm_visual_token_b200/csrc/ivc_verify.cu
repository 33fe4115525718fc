// ivc_verify.cu — drafted trees against the target's probabilities.
//
// The walk (definition in ivc.h) tries a node's children in ascending order, and
// parents stand before their children, so the whole walk is one ascending scan:
// node j is tried iff its parent is the current node when the scan reaches it.
// Its tests need two probabilities per node, which are gathered up front; only a
// rejection with draft probabilities needs a pass over the vocabulary, for the sum
// of max(r / z - q / w, 0), and the final draw one over the row it ends in (none
// when its last rejection just made that pass).
//
// r is a function of the row's fp32 inputs and the scalars z_i, w_i, c_i of the
// node's rejections so far, so every pass recomputes it in fp64 from the inputs, with
// the formula's roundings: nothing is stored. The n-th rejection at a node repeats the
// n - 1 before it for every value, so a node costs the square of its rejections: a
// star of 128 nodes over 151001 tokens that are all rejected takes 7.5 ms. Sums are
// fp64 in a fixed order (per lane, warp, slice), which is not the order of the tokens:
// results are the same from call to call, and the formula's up to the rounding of sums.
//
// A sequence is one cluster of 8 CTAs: each walks for itself (the same scalars) and
// sums a contiguous eighth of the vocabulary, and the eight sums are exchanged
// through distributed shared memory. One sequence without a rejection is bound by
// its chain of dependent loads (offsets, tokens, probabilities, row): 6.8 us for 151001
// tokens. A rejection with draft probabilities adds a pass, bound by the fp64 and
// conversion pipes of the cluster's SMs: 7 rejections of one node 57 us, 15 of them
// 169 us. A batch takes as long as its longest chain of them, and 48 sequences'
// clusters do not fit at once: 48 trees of 16 nodes 49 to 62 us by their inputs,
// without drafts 17 us (their rows in one read from HBM would be 4), with 15 rejections
// of the root each 435 us. (Device times over changing inputs.)
// 384 threads of 80 registers: 512 threads spill, 256 were a sixth slower for one
// sequence. Clusters of 16 halve a pass but fewer fit: for the trees a twentieth
// faster, without rejections a fifth slower.
#include <cuda_runtime.h>

#include "ivc_internal.h"
#include "ivc_ptx.cuh"

namespace ivc {
namespace {

constexpr int VF_THREADS = 384;
constexpr int VF_WARPS = VF_THREADS / 32;
constexpr int VF_CLUSTER = 8;
// A vocabulary up to this size is one CTA's: for 4096 tokens one sequence takes 4.1 us
// (a cluster 4.8), with 7 rejections 21.6 (20.2), 48 of those 21.8 (37.9); for 8192 tokens
// 4.6 (4.8), 26.7 (20.7) and 27.1 (38.8).
constexpr int VF_SMALL = 4096;
constexpr int VF_BATCH = 8;     // values a thread has in flight

struct VerifyArgs {
  const float* p;
  long long p_ld;
  const float* q;
  long long q_ld;
  int N, V, B;
  const int32_t* tokens;
  const int32_t* parents;
  const int32_t* offsets;
  const float* u;
  const float* u_next;
  int32_t* path;
  int path_stride;
  int32_t* n_path;
  int32_t* next_token;
  int* status;
};

__device__ __forceinline__ double positive(float x) { return static_cast<double>(fmaxf(x, 0.f)); }

// The rejections at the current node.
struct Rejected {
  double iz[IVC_MAX_TREE], iw[IVC_MAX_TREE];  // 1 / z, 1 / w before rejection i
  int token[IVC_MAX_TREE];
  int n;
};

// max(x, 0) without the fp64 comparison: x is no NaN (or the row has infinities
// and its sum is refused).
__device__ __forceinline__ double above_zero(double x) {
  const int hi = __double2hiint(x), keep = ~(hi >> 31);
  return __hiloint2double(hi & keep, __double2loint(x) & keep);
}

// r / z - q / w as the formula has it: both products rounded. Fused, one of them would
// not be, and where the two are equal (all that is left of the draft is left of the
// target, and a sibling repeats a rejected token) the remainder would be 1e-17 of
// noise instead of 0: more siblings tried, and the next token drawn from the noise.
__device__ __forceinline__ double less(double r, double iz, double q, double iw) {
  return __dsub_rn(__dmul_rn(r, iz), __dmul_rn(q, iw));
}

// VF_BATCH tokens v0, v0 + step, ... below `end`: their inputs (0 for the others) ...
struct Batch {
  float p[VF_BATCH], q[VF_BATCH];
};
__device__ __forceinline__ void fetch(const float* p, const float* q, int v0, int step, int end,
                                      Batch& x) {
#pragma unroll
  for (int e = 0; e < VF_BATCH; ++e) {
    const int v = v0 + e * step;
    x.p[e] = v < end ? p[v] : 0.f;
    x.q[e] = q != nullptr && v < end ? q[v] : 0.f;
  }
}
// ... and their r after the node's rejections. With draft probabilities a rejected
// token needs no exclusion from q here: u q(c) / w >= r(c) / z with u < 1 makes
// its r 0, and so it stays.
__device__ __forceinline__ void left_of(const Batch& x, bool dense, int v0, int step,
                                        const Rejected& rj, double (&r)[VF_BATCH]) {
  const int n = rj.n;
  if (dense) {
    double d[VF_BATCH];
#pragma unroll
    for (int e = 0; e < VF_BATCH; ++e) {
      d[e] = positive(x.q[e]);
      r[e] = above_zero(positive(x.p[e]) - d[e]);  // the first rejection: z = w = 1
    }
    for (int i = 1; i < n; ++i) {
      const double iz = rj.iz[i], iw = rj.iw[i];
#pragma unroll
      for (int e = 0; e < VF_BATCH; ++e) r[e] = above_zero(less(r[e], iz, d[e], iw));
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < VF_BATCH; ++e) r[e] = positive(x.p[e]);
  for (int i = 0; i < n; ++i) {
    const int tok = rj.token[i];
#pragma unroll
    for (int e = 0; e < VF_BATCH; ++e)
      if (v0 + e * step == tok) r[e] = 0.0;
  }
}

// What the CTAs of a cluster tell each other: the sum of their slice, double
// buffered by pass.
struct Sums {
  double slice[2][VF_CLUSTER];
};

// This CTA's sum into every CTA of the cluster, and all of them back.
template <int CL>
__device__ void exchange(Sums& sums, int pass, double mine) {
  if (CL == 1) {
    if (threadIdx.x == 0) sums.slice[pass & 1][0] = mine;
    __syncthreads();
    return;
  }
  if (threadIdx.x < CL) {
    const uint32_t local = smem_u32(&sums.slice[pass & 1][cluster_ctarank()]);
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(threadIdx.x));
    asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(remote), "d"(mine) : "memory");
  }
  cluster_sync();
}

template <int CL>
__global__ void __launch_bounds__(VF_THREADS, 2)
    verify_kernel(const __grid_constant__ VerifyArgs a) {
  __shared__ Rejected rj;
  __shared__ Sums sums;
  __shared__ double s_seg[VF_WARPS];  // sums of the warps' segments of the slice
  __shared__ double s_scan[VF_WARPS];
  __shared__ int s_tok[IVC_MAX_TREE], s_par[IVC_MAX_TREE];
  __shared__ float s_u[IVC_MAX_TREE], s_p[IVC_MAX_TREE], s_q[IVC_MAX_TREE];
  __shared__ int s_hit, s_last;
  if (CL > 1) cluster_sync();  // every CTA of the cluster runs: its shared memory may be written
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x / CL, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = CL == 1 ? 0 : static_cast<int>(cluster_ctarank());
  int32_t* path = a.path + static_cast<size_t>(b) * a.path_stride;
  const int first = a.offsets[b], n = a.offsets[b + 1] - first;
  const bool bad = first < 0 || n < 0 || n > IVC_MAX_TREE || first > a.N - n;
  if (bad || n == 0) {  // the same in every CTA of the cluster
    if (rank == 0) {
      for (int i = tid; i < a.path_stride; i += VF_THREADS) path[i] = -1;
      if (tid == 0) {
        if (bad) atomicOr(a.status, DEV_BAD_TREE);
        a.n_path[b] = 0;
        a.next_token[b] = -1;
      }
    }
    return;
  }
  if (tid < n) {
    int par = a.parents ? a.parents[first + tid] : tid - 1;
    int tok = a.tokens[first + tid];
    s_u[tid] = a.u[first + tid];
    int flags = 0;
    if (par < -1 || par >= tid) {
      flags |= DEV_BAD_TREE;
      par = -1;
    }
    if (tid > 0 && (tok < 0 || tok >= a.V)) {
      flags |= DEV_BAD_PROBS;
      tok = -1;
    }
    if (flags && rank == 0) atomicOr(a.status, flags);
    s_par[tid] = par;
    s_tok[tid] = tok;
    if (par >= 0 && tok >= 0) {
      s_p[tid] = a.p[static_cast<long long>(first + par) * a.p_ld + tok];
      s_q[tid] = a.q ? a.q[static_cast<long long>(first + par) * a.q_ld + tok] : 1.f;
    }
  }
  if (tid == 0) rj.n = 0;
  __syncthreads();

  // this CTA's slice of the vocabulary, and the warp's segment of it
  const int slice = (a.V + CL - 1) / CL;
  const int lo = min(a.V, rank * slice), hi = min(a.V, lo + slice);
  const int seg = (slice + VF_WARPS - 1) / VF_WARPS;
  const int s0 = min(hi, lo + warp * seg), s1 = min(hi, s0 + seg);

  const float* p = a.p + static_cast<long long>(first) * a.p_ld;
  const float* q = a.q ? a.q + static_cast<long long>(first) * a.q_ld : nullptr;
  int passes = 0;
  bool summed = false;  // s_seg and sums hold the current r
  // the sum of r: per segment, per slice, in all
  auto sum_all = [&]() -> double {
    double acc[2] = {0.0, 0.0};
    const float* qq = rj.n > 0 ? q : nullptr;
    for (int v = s0 + lane; v < s1; v += 32 * VF_BATCH) {
      Batch x;
      fetch(p, qq, v, 32, s1, x);
      double r[VF_BATCH];
      left_of(x, qq != nullptr, v, 32, rj, r);
#pragma unroll
      for (int e = 0; e < VF_BATCH; ++e) acc[e & 1] += r[e];
    }
    double x = acc[0] + acc[1];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (lane == 0) s_seg[warp] = x;
    __syncthreads();
    double mine = 0.0;
#pragma unroll
    for (int w = 0; w < VF_WARPS; ++w) mine += s_seg[w];
    exchange<CL>(sums, passes, mine);
    double all = 0.0;
#pragma unroll
    for (int k = 0; k < CL; ++k) all += sums.slice[passes & 1][k];
    ++passes;
    summed = true;
    return all;
  };

  // the walk: the same in every thread
  int cur = 0, count = 1;
  double z = 1.0, w = 1.0;
  if (rank == 0 && tid == 0) path[0] = 0;
  for (int j = 1; j < n && count < a.path_stride; ++j) {
    const int tok = s_tok[j];
    if (s_par[j] != cur || !(z > 0.0) || tok < 0) continue;
    double r = positive(s_p[j]), d = q != nullptr ? positive(s_q[j]) : 1.0;
    for (int i = 0; i < rj.n; ++i) {
      if (q != nullptr) {
        r = less(r, rj.iz[i], d, rj.iw[i]);
        r = r > 0.0 ? r : 0.0;
      }
      if (rj.token[i] == tok) {
        if (q != nullptr) d = 0.0;
        else r = 0.0;
      }
    }
    const bool stands = static_cast<double>(s_u[j]) * d * z < r * w;
    __syncthreads();  // rj is read
    if (stands) {
      cur = j;
      p = a.p + static_cast<long long>(first + j) * a.p_ld;
      if (q != nullptr) q = a.q + static_cast<long long>(first + j) * a.q_ld;
      z = w = 1.0;
      summed = false;
      if (tid == 0) {
        rj.n = 0;
        if (rank == 0) path[count] = j;
      }
      ++count;
      __syncthreads();
    } else {
      if (tid == 0) {
        const int k = rj.n;
        rj.iz[k] = 1.0 / z;
        rj.iw[k] = w > 0.0 ? 1.0 / w : 0.0;
        rj.token[k] = tok;
        rj.n = k + 1;
      }
      __syncthreads();
      if (q != nullptr) {
        z = sum_all();
        w -= d;
      } else {
        z -= r;
        summed = false;
      }
    }
  }

  // the draw
  double total = summed ? z : sum_all();
  if (!(total > 0.0) && rj.n > 0) {  // nothing left: the node's own row
    __syncthreads();
    if (tid == 0) rj.n = 0;
    __syncthreads();
    total = sum_all();
  }
  if (rank == 0) {
    for (int i = count + tid; i < a.path_stride; i += VF_THREADS) path[i] = -1;
    if (tid == 0) a.n_path[b] = count;
  }
  if (!(total > 0.0) || isinf(total)) {
    if (rank == 0 && tid == 0) {
      atomicOr(a.status, DEV_BAD_PROBS);
      a.next_token[b] = -1;
    }
    return;
  }
  // the slice, then the segment, in which the running sum passes the goal; where
  // rounding leaves none, the last one that holds anything
  const double goal = static_cast<double>(a.u_next[b]) * total;
  const double* slices = sums.slice[(passes - 1) & 1];
  double base = 0.0, run = 0.0;
  int owner = -1, last = 0;
#pragma unroll
  for (int k = 0; k < CL; ++k) {
    const double next = run + slices[k];
    if (slices[k] > 0.0) {
      if (owner < 0) { last = k; base = run; }
      if (owner < 0 && next > goal) owner = k;
    }
    run = next;
  }
  if (owner < 0) owner = last;
  if (rank != owner) return;
  run = base;
  int part = -1;
  last = 0;
  for (int k = 0; k < VF_WARPS; ++k) {
    const double next = run + s_seg[k];
    if (s_seg[k] > 0.0) {
      if (part < 0) { last = k; base = run; }
      if (part < 0 && next > goal) part = k;
    }
    run = next;
  }
  if (part < 0) part = last;
  // that segment once more, in thread order: VF_BATCH neighbouring values each
  if (tid == 0) { s_hit = a.V; s_last = -1; }
  const int e0 = lo + part * seg, e1 = min(hi, e0 + seg);
  run = base;
  for (int v0 = e0; v0 < e1; v0 += VF_THREADS * VF_BATCH) {
    const int v = v0 + tid * VF_BATCH;
    const float* qq = rj.n > 0 ? q : nullptr;
    Batch x;
    fetch(p, qq, v, 1, e1, x);
    double r[VF_BATCH], mine = 0.0;
    left_of(x, qq != nullptr, v, 1, rj, r);
#pragma unroll
    for (int e = 0; e < VF_BATCH; ++e) mine += r[e];
    double incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    __syncthreads();
    if (lane == 31) s_scan[warp] = incl;
    __syncthreads();
    double before = run + incl - mine;
    for (int k = 0; k < VF_WARPS; ++k) {
      if (k < warp) before += s_scan[k];
      run += s_scan[k];
    }
#pragma unroll
    for (int e = 0; e < VF_BATCH; ++e) {
      before += r[e];
      if (r[e] > 0.0) {
        atomicMax(&s_last, v + e);
        if (before > goal) atomicMin(&s_hit, v + e);
      }
    }
  }
  __syncthreads();
  if (tid == 0) a.next_token[b] = s_hit < a.V ? s_hit : s_last;
}

}  // namespace
}  // namespace ivc

using namespace ivc;

extern "C" int ivc_verify_drafts(const float* p, long long p_ld, const float* q, long long q_ld,
                                 int N, int V, const int32_t* tokens, const int32_t* parents,
                                 const int32_t* offsets, int B, const float* u,
                                 const float* u_next, int32_t* path, int path_stride,
                                 int32_t* n_path, int32_t* next_token, void* workspace,
                                 size_t ws_bytes, ivc_stream_t stream) {
  if (N < 0 || V < 1 || B < 0 || path_stride < 1) return IVC_EINVAL;
  if (p_ld < V || (q && q_ld < V)) return IVC_EINVAL;
  if (B > (1 << 24) || V > (1 << 28)) return IVC_EUNSUPPORTED;
  if (B > 0 && (!offsets || !u_next || !path || !n_path || !next_token)) return IVC_EINVAL;
  if (N > 0 && (!p || !tokens || !u)) return IVC_EINVAL;
  if (const int rc = step_ws_ok(workspace, ws_bytes, IVC_STEP_WORKSPACE_BYTES)) return rc;
  if (B == 0) return IVC_OK;
  const VerifyArgs a{p, p_ld, q, q_ld, N, V, B, tokens, parents, offsets, u, u_next,
                     path, path_stride, n_path, next_token, static_cast<int*>(workspace)};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  TraceScope ts("verify_drafts", s);
  if (V <= VF_SMALL) return launch_k(verify_kernel<1>, dim3(B), dim3(VF_THREADS), 0, s, 1, a);
  return launch_k(verify_kernel<VF_CLUSTER>, dim3(static_cast<unsigned>(B) * VF_CLUSTER),
                  dim3(VF_THREADS), 0, s, VF_CLUSTER, a);
}
