// ivc_tree_attend.cu — attention of drafted trees over the paged cache.
//
// out_i = sum_j softmax_j(scale q_i . k_j) v_j over the committed tokens, the
// node's ancestors and the node itself. One pass with the running maximum m and
// sum l: per 128 keys m' = max(m, max s), l' = l e^(m - m') + sum e^(s - m'),
// o' = o e^(m - m') + sum e^(s - m') v; out = o / l.
//
// A CTA takes one (node, query head): thread t scores key t of a tile, then
// accumulates value column t. Keys that the node does not see are skipped, not
// multiplied by zero, so what stands in them has no influence.
#include <cuda_runtime.h>

#include "ivc_internal.h"
#include "ivc_ptx.cuh"

namespace ivc {
namespace {

constexpr int TA_KEYS = 128;

struct TreeArgs {
  const bf16* q;
  long long q_ld;
  int N, q_heads, layer, B;
  float scale;
  const int32_t* parents;
  const int32_t* offsets;
  const int32_t* seqs;
  bf16* out;
  int* status;
};

template <int D>
__global__ void __launch_bounds__(TA_KEYS)
    tree_attend_kernel(const __grid_constant__ ivc_cache c, const __grid_constant__ TreeArgs a) {
  __shared__ float s_q[D], s_p[TA_KEYS], s_red[TA_KEYS / 32];
  __shared__ uint8_t s_sees[IVC_MAX_TREE];
  __shared__ long long s_row[TA_KEYS];
  pdl_wait();
  pdl_trigger();
  const int row = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
  if (row == 0 && h == 0)
    for (int b = tid; b < a.B; b += TA_KEYS)
      if (a.offsets[b + 1] < a.offsets[b] || a.offsets[b + 1] > a.N) atomicOr(a.status, DEV_BAD_TREE);
  if (row >= a.offsets[a.B]) return;
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.offsets[mid] <= row) lo = mid; else hi = mid;
  }
  const int first = a.offsets[lo], n = a.offsets[lo + 1] - first;
  const int s = a.seqs ? a.seqs[lo] : lo;
  if (first < 0 || first > row || n > IVC_MAX_TREE || first + n > a.N || row - first >= n) {
    if (tid == 0) atomicOr(a.status, DEV_BAD_TREE);
    return;
  }
  if (s < 0 || s >= c.max_seqs || c.length[s] < 0 || c.n_pages[s] > c.max_pages ||
      static_cast<long long>(c.length[s]) + n > static_cast<long long>(c.n_pages[s]) * c.page_tokens) {
    if (tid == 0) atomicOr(a.status, DEV_BAD_CACHE);
    return;
  }
  const int len = c.length[s], node = row - first;
  s_sees[tid] = 0;
  for (int d = tid; d < D; d += TA_KEYS)
    s_q[d] = __bfloat162float(a.q[static_cast<long long>(row) * a.q_ld + h * D + d]);
  __syncthreads();
  if (tid == 0) {
    for (int i = node; i >= 0;) {
      s_sees[i] = 1;
      const int par = a.parents ? a.parents[first + i] : i - 1;
      if (par < -1 || par >= i) {
        atomicOr(a.status, DEV_BAD_TREE);
        break;
      }
      i = par;
    }
  }
  __syncthreads();
  const int kvh = h / (a.q_heads / c.kv_heads);
  const bf16* kb = static_cast<const bf16*>(c.k);
  const bf16* vb = static_cast<const bf16*>(c.v);
  const int32_t* table = c.table + static_cast<size_t>(s) * c.max_pages;
  float m = -INFINITY, l = 0.f, o = 0.f;
  for (int t0 = 0; t0 < len + n; t0 += TA_KEYS) {
    const int t = t0 + tid;
    float x = -INFINITY;
    bool sees = t < len || (t < len + n && s_sees[t - len]);
    long long at = -1;
    if (sees) {
      const int page = table[t / c.page_tokens];
      if (page >= 0 && page < c.pages)
        at = ((static_cast<long long>(a.layer) * c.pages + page) * c.kv_heads + kvh) *
                 c.page_tokens * D + static_cast<long long>(t % c.page_tokens) * D;
      else
        atomicOr(a.status, DEV_BAD_CACHE);
      if (at >= 0) {
        x = 0.f;
        for (int d = 0; d < D; ++d) x += s_q[d] * __bfloat162float(kb[at + d]);
        x *= a.scale;
      }
    }
    s_row[tid] = at;
    float v = x;
#pragma unroll
    for (int e = 16; e > 0; e >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, e));
    if ((tid & 31) == 0) s_red[tid >> 5] = v;
    __syncthreads();
    const float m2 = fmaxf(m, fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3])));
    const float base = m2 == -INFINITY ? 0.f : m2;
    const float f = expf(m - base);
    s_p[tid] = at >= 0 ? expf(x - base) : 0.f;
    __syncthreads();
    l *= f;
    o *= f;
    for (int j = 0; j < TA_KEYS; ++j) {
      if (s_row[j] < 0) continue;
      l += s_p[j];
      if (tid < D) o += s_p[j] * __bfloat162float(vb[s_row[j] + tid]);
    }
    m = m2;
    __syncthreads();
  }
  if (tid < D)
    a.out[(static_cast<long long>(row) * a.q_heads + h) * D + tid] = __float2bfloat16_rn(o / l);
}

}  // namespace
}  // namespace ivc

using namespace ivc;

extern "C" {

size_t ivc_tree_attention_workspace_size(const ivc_cache* c, int N, int q_heads, int B) {
  if (cache_ok(c) != IVC_OK || N < 0 || B < 0 || q_heads < 1) return 0;
  return IVC_STEP_WORKSPACE_BYTES;
}

int ivc_tree_attention(const ivc_cache* c, int layer, const void* q, long long q_ld, int N,
                       int q_heads, float scale, const int32_t* parents, const int32_t* offsets,
                       const int32_t* seqs, int B, void* out, void* workspace, size_t ws_bytes,
                       ivc_stream_t stream) {
  if (const int rc = cache_ok(c)) return rc;
  if (layer < 0 || layer >= c->layers || N < 0 || B < 0 || q_heads < 1) return IVC_EINVAL;
  if (!(scale > -INFINITY && scale < INFINITY)) return IVC_EINVAL;
  if (q_heads % c->kv_heads != 0 || q_heads / c->kv_heads > 64 || B > 4096) return IVC_EUNSUPPORTED;
  if (q_ld % 8 != 0 || q_ld < static_cast<long long>(q_heads) * c->head_dim) return IVC_EUNSUPPORTED;
  if (!offsets || (N > 0 && (!q || !out))) return IVC_EINVAL;
  auto al = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  if (!al(q) || !al(out)) return IVC_EALIGN;
  if (const int rc = step_ws_ok(workspace, ws_bytes,
                                ivc_tree_attention_workspace_size(c, N, q_heads, B)))
    return rc;
  if (N == 0 || B == 0) return IVC_OK;
  const TreeArgs a{static_cast<const bf16*>(q), q_ld, N, q_heads, layer, B, scale, parents, offsets,
                   seqs, static_cast<bf16*>(out), static_cast<int*>(workspace)};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  TraceScope ts("tree_attention", s);
  return launch_k(c->head_dim == 64 ? tree_attend_kernel<64> : tree_attend_kernel<128>,
                  dim3(N, q_heads), dim3(TA_KEYS), 0, s, 1, *c, a);
}

}  // extern "C"
