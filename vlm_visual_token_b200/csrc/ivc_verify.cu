// ivc_verify.cu — drafted trees against the target's probabilities.
//
// The walk (definition in ivc.h) tries a node's children in ascending order, and
// parents stand before their children, so the whole walk is one ascending scan:
// node j is tried iff its parent is the current node when the scan reaches it.
// A test needs two probabilities, which are gathered up front; only a rejection
// with draft probabilities needs a pass over the vocabulary, for the sum of
// max(r / z - q / w, 0), and the final draw one over the row it ends in.
//
// r is a function of the row's fp32 inputs and the scalars z_i, w_i, c_i of the
// node's rejections so far, so every pass recomputes it in fp64 from the
// inputs: nothing is stored and nothing rounded in between. Sums are fp64 in a
// fixed order.
#include <cuda_runtime.h>

#include "ivc_internal.h"
#include "ivc_ptx.cuh"

namespace ivc {
namespace {

constexpr int VF_THREADS = 1024;

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

__device__ __forceinline__ double positive(float x) { return x > 0.f ? static_cast<double>(x) : 0.0; }

// The rejections at the current node.
struct Rejected {
  double iz[IVC_MAX_TREE], iw[IVC_MAX_TREE];  // 1 / z, 1 / w before rejection i
  int token[IVC_MAX_TREE];
  int n;
};

// r(v) after the node's rejections. DENSE: with draft probabilities.
__device__ __forceinline__ double left_of(const float* p, const float* q, int v, const Rejected& rj) {
  double r = positive(p[v]);
  if (q != nullptr) {
    if (rj.n == 0) return r;
    double d = positive(q[v]);
    for (int i = 0; i < rj.n; ++i) {
      r = fmax(r * rj.iz[i] - d * rj.iw[i], 0.0);
      if (v == rj.token[i]) d = 0.0;
    }
  } else {
    for (int i = 0; i < rj.n; ++i)
      if (v == rj.token[i]) r = 0.0;
  }
  return r;
}

__device__ double block_sum(double x, double* s_warp) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  __syncthreads();
  if (lane == 0) s_warp[warp] = x;
  __syncthreads();
  double sum = 0.0;
  for (int i = 0; i < VF_THREADS / 32; ++i) sum += s_warp[i];
  return sum;
}

__global__ void __launch_bounds__(VF_THREADS) verify_kernel(const __grid_constant__ VerifyArgs a) {
  __shared__ Rejected rj;
  __shared__ double s_warp[32];
  __shared__ int s_tok[IVC_MAX_TREE], s_par[IVC_MAX_TREE];
  __shared__ float s_u[IVC_MAX_TREE];
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x, tid = threadIdx.x;
  int32_t* path = a.path + static_cast<size_t>(b) * a.path_stride;
  const int first = a.offsets[b], n = a.offsets[b + 1] - first;
  for (int i = tid; i < a.path_stride; i += VF_THREADS) path[i] = -1;
  if (first < 0 || n < 0 || n > IVC_MAX_TREE || first > a.N - n) {
    if (tid == 0) atomicOr(a.status, DEV_BAD_TREE);
  }
  if (n < 1 || first < 0 || n > IVC_MAX_TREE || first > a.N - n) {
    if (tid == 0) {
      a.n_path[b] = 0;
      a.next_token[b] = -1;
    }
    return;
  }
  if (tid < n) {
    int par = a.parents ? a.parents[first + tid] : tid - 1;
    if (par < -1 || par >= tid) {
      atomicOr(a.status, DEV_BAD_TREE);
      par = -1;
    }
    s_par[tid] = par;
    int tok = a.tokens[first + tid];
    if (tid > 0 && (tok < 0 || tok >= a.V)) {
      atomicOr(a.status, DEV_BAD_PROBS);
      tok = -1;
    }
    s_tok[tid] = tok;
    s_u[tid] = a.u[first + tid];
  }
  if (tid == 0) rj.n = 0;
  __syncthreads();

  const float* p = a.p + static_cast<long long>(first) * a.p_ld;
  const float* q = a.q ? a.q + static_cast<long long>(first) * a.q_ld : nullptr;
  int cur = 0, count = 1;
  double z = 1.0, w = 1.0;
  if (tid == 0) path[0] = 0;
  for (int j = 1; j < n && count < a.path_stride; ++j) {
    if (s_par[j] != cur || !(z > 0.0) || s_tok[j] < 0) continue;
    const int tok = s_tok[j];
    const double r = left_of(p, q, tok, rj);
    double d = 1.0;
    if (q != nullptr) {
      d = positive(q[tok]);
      for (int i = 0; i < rj.n; ++i)
        if (rj.token[i] == tok) d = 0.0;
    }
    if (static_cast<double>(s_u[j]) * d * z < r * w) {
      cur = j;
      p = a.p + static_cast<long long>(first + j) * a.p_ld;
      if (q != nullptr) q = a.q + static_cast<long long>(first + j) * a.q_ld;
      z = w = 1.0;
      if (tid == 0) path[count] = j;
      ++count;
      __syncthreads();
      if (tid == 0) rj.n = 0;
      __syncthreads();
    } else {
      __syncthreads();
      if (tid == 0) {
        rj.iz[rj.n] = 1.0 / z;
        rj.iw[rj.n] = w > 0.0 ? 1.0 / w : 0.0;
        rj.token[rj.n] = tok;
        ++rj.n;
      }
      __syncthreads();
      if (q != nullptr) {
        double sum = 0.0;
        for (int v = tid; v < a.V; v += VF_THREADS) sum += left_of(p, q, v, rj);
        z = block_sum(sum, s_warp);
        w -= d;
      } else {
        z -= r;
      }
    }
  }

  // the draw: contiguous slices of the row per thread
  const int per = (a.V + VF_THREADS - 1) / VF_THREADS;
  const int v0 = min(a.V, tid * per), v1 = min(a.V, v0 + per);
  for (int pass = 0; pass < 2; ++pass) {
    double mine = 0.0;
    for (int v = v0; v < v1; ++v) mine += left_of(p, q, v, rj);
    const double total = block_sum(mine, s_warp);
    if (!(total > 0.0) && pass == 0 && rj.n > 0) {  // nothing left: the node's own row
      __syncthreads();
      if (tid == 0) rj.n = 0;
      __syncthreads();
      continue;
    }
    int token = -1;
    if (total > 0.0 && !isinf(total)) {
      // exclusive sums in thread order
      __shared__ double s_sum[VF_THREADS];
      s_sum[tid] = mine;

      __syncthreads();
      if (tid == 0) {
        double t = 0.0;
        for (int i = 0; i < VF_THREADS; ++i) {
          const double m = s_sum[i];
          s_sum[i] = t;
          t += m;
        }
        const double goal = static_cast<double>(a.u_next[b]) * t;
        s_warp[0] = goal;
      }
      __syncthreads();
      const double goal = s_warp[0];
      double t = s_sum[tid];
      int last = -1, hit = -1;
      for (int v = v0; v < v1; ++v) {
        const double r = left_of(p, q, v, rj);
        t += r;
        if (r > 0.0) {
          last = v;
          if (hit < 0 && t > goal) hit = v;
        }
      }
      // the least hit, or (a goal that rounding put at the sum) the last value
      __shared__ int s_hit, s_last;
      if (tid == 0) { s_hit = a.V; s_last = -1; }
      __syncthreads();
      if (hit >= 0) atomicMin(&s_hit, hit);
      if (last >= 0) atomicMax(&s_last, last);
      __syncthreads();
      token = s_hit < a.V ? s_hit : s_last;
    }
    if (tid == 0) {
      if (token < 0) atomicOr(a.status, DEV_BAD_PROBS);
      a.next_token[b] = token;
      a.n_path[b] = count;
    }
    break;
  }
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
  if (B > 0 && (!offsets || !u_next || !path || !n_path || !next_token)) return IVC_EINVAL;
  if (N > 0 && (!p || !tokens || !u)) return IVC_EINVAL;
  if (const int rc = step_ws_ok(workspace, ws_bytes, IVC_STEP_WORKSPACE_BYTES)) return rc;
  if (B == 0) return IVC_OK;
  const VerifyArgs a{p, p_ld, q, q_ld, N, V, B, tokens, parents, offsets, u, u_next,
                     path, path_stride, n_path, next_token, static_cast<int*>(workspace)};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  TraceScope ts("verify_drafts", s);
  return launch_k(verify_kernel, dim3(B), dim3(VF_THREADS), 0, s, 1, a);
}
