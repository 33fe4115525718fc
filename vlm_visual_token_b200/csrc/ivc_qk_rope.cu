// ivc_qk_rope.cu — per-head norms of queries and keys, position rotation and
// storage of keys and values in the cache's pages, in one pass.
//
// Per token and head x of D values, in fp32 (statistics and products) from the
// bf16 projections:
//   y = x rsqrt(mean(x^2) + eps) gamma,
//   out_j = y_j cos(t f_j) - y_{j+D/2} sin(t f_j),
//   out_{j+D/2} = y_{j+D/2} cos(t f_j) + y_j sin(t f_j),  f_j = theta^(-2j/D),
// rounded to bf16 once. The turn t f_j / 2 pi is formed and reduced to
// [-1/2, 1/2] in fp64 (a far position times a frequency in fp32 is off by
// t * 2^-24 radians: 0.002 at t = 40960, the size of a bf16 rounding), then
// sincospif in fp32. A token's D/2 rotations are computed once and serve all
// of its heads.
//
// Bound by HBM (each value is read and written once). A CTA takes one token: 8
// bf16 per lane, D/8 lanes per head, so a head's sum of squares and its other
// half's values are exchanged by shuffles; all 16-byte loads of a thread are
// issued before the first is used.
#include <cuda_runtime.h>

#include <cmath>

#include "ivc_internal.h"
#include "ivc_ptx.cuh"

namespace ivc {
namespace {

constexpr int QR_THREADS = 256;
constexpr int QR_LOADS = 4;  // heads a thread holds at a time

struct RopeFreq {
  double turn[64];  // f_j / (2 pi)
};

struct QkArgs {
  const bf16* qkv;
  long long ld;
  int N, q_heads, layer, B;
  const bf16* gamma_q;
  const bf16* gamma_k;
  float eps;
  const int32_t* positions;
  const int32_t* offsets;
  const int32_t* seqs;
  bf16* q_out;
  int* status;
};

__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int D>
__global__ void __launch_bounds__(QR_THREADS)
    qk_norm_rope_kernel(const __grid_constant__ ivc_cache c, const __grid_constant__ QkArgs a,
                        const __grid_constant__ RopeFreq freq) {
  constexpr int LANES = D / 8;                      // lanes per head
  constexpr int AT_ONCE = QR_THREADS / LANES;       // heads per pass of the CTA
  __shared__ float s_cos[D / 2], s_sin[D / 2];
  __shared__ long long s_row;                       // first value of the token in its page, or -1
  pdl_wait();
  pdl_trigger();
  const int tok = blockIdx.x;
  if (tok == 0) {
    for (int b = threadIdx.x; b < a.B; b += QR_THREADS)
      if (a.offsets[b + 1] < a.offsets[b] || a.offsets[b + 1] > a.N) atomicOr(a.status, DEV_BAD_TREE);
    if (threadIdx.x == 0 && a.offsets[0] != 0) atomicOr(a.status, DEV_BAD_TREE);
  }
  if (tok >= a.offsets[a.B]) return;  // behind the last sequence
  if (threadIdx.x < D / 2) {
    double t = a.positions[tok] * freq.turn[threadIdx.x];
    t -= rint(t);
    float sn, cs;
    sincospif(static_cast<float>(2.0 * t), &sn, &cs);
    s_cos[threadIdx.x] = cs;
    s_sin[threadIdx.x] = sn;
  } else if (threadIdx.x == QR_THREADS - 1) {
    // the sequence that row tok belongs to: the last one that starts at or before it
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.offsets[mid] <= tok) lo = mid; else hi = mid;
    }
    const int s = a.seqs ? a.seqs[lo] : lo;
    long long row = -1;
    if (s >= 0 && s < c.max_seqs && a.offsets[lo] <= tok) {
      const long long pos = static_cast<long long>(c.length[s]) + tok - a.offsets[lo];
      const int np = min(c.n_pages[s], c.max_pages);
      if (pos >= 0 && pos < static_cast<long long>(np) * c.page_tokens) {
        const int page = c.table[static_cast<size_t>(s) * c.max_pages + pos / c.page_tokens];
        if (page >= 0 && page < c.pages)
          row = ((static_cast<long long>(a.layer) * c.pages + page) * c.kv_heads *
                     c.page_tokens + pos % c.page_tokens) * D;
      }
    }
    if (row < 0) atomicOr(a.status, DEV_BAD_CACHE);
    s_row = row;
  }
  __syncthreads();
  const int lane = threadIdx.x % LANES;
  const bool upper = lane >= LANES / 2;             // the second half of the head
  const int j0 = (lane % (LANES / 2)) * 8;          // its rotations
  const int heads = a.q_heads + 2 * c.kv_heads;
  const bf16* src = a.qkv + static_cast<long long>(tok) * a.ld + lane * 8;
  const long long head_stride = static_cast<long long>(c.page_tokens) * D;
  for (int h0 = threadIdx.x / LANES; h0 < (heads + AT_ONCE - 1) / AT_ONCE * AT_ONCE;
       h0 += AT_ONCE * QR_LOADS) {
    uint4 u[QR_LOADS];
#pragma unroll
    for (int k = 0; k < QR_LOADS; ++k) {
      const int h = h0 + k * AT_ONCE;
      u[k] = h < heads ? *reinterpret_cast<const uint4*>(src + static_cast<long long>(h) * D)
                       : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int k = 0; k < QR_LOADS; ++k) {
      const int h = h0 + k * AT_ONCE;
      float x[8], other[8];
      unpack8(u[k], x);
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss += x[i] * x[i];
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const bool is_q = h < a.q_heads;
      if (h < a.q_heads + c.kv_heads) {
        float g[8];
        unpack8(*reinterpret_cast<const uint4*>((is_q ? a.gamma_q : a.gamma_k) + lane * 8), g);
        const float r = 1.f / sqrtf(ss * (1.f / D) + a.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] * r * g[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) other[i] = __shfl_xor_sync(0xffffffffu, x[i], LANES / 2);
      if (h >= heads) continue;
      if (h < a.q_heads + c.kv_heads) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float cs = s_cos[j0 + i], sn = upper ? s_sin[j0 + i] : -s_sin[j0 + i];
          x[i] = x[i] * cs + other[i] * sn;
        }
        u[k] = pack8(x);
      }
      if (is_q) {
        *reinterpret_cast<uint4*>(a.q_out +
                                  (static_cast<long long>(tok) * a.q_heads + h) * D + lane * 8) = u[k];
      } else if (s_row >= 0) {
        const int kv = h - a.q_heads;
        bf16* page = static_cast<bf16*>(kv < c.kv_heads ? c.k : c.v);
        *reinterpret_cast<uint4*>(page + s_row + (kv % c.kv_heads) * head_stride + lane * 8) = u[k];
      }
    }
  }
}

}  // namespace
}  // namespace ivc

using namespace ivc;

extern "C" int ivc_qk_norm_rope(const ivc_cache* c, int layer, const void* qkv, long long ld, int N,
                                int q_heads, const void* q_gamma, const void* k_gamma, float eps,
                                double theta, const int32_t* positions, const int32_t* offsets,
                                const int32_t* seqs, int B, void* q_out, void* workspace,
                                size_t ws_bytes, ivc_stream_t stream) {
  if (const int rc = cache_ok(c)) return rc;
  if (layer < 0 || layer >= c->layers || N < 0 || B < 0 || q_heads < 1) return IVC_EINVAL;
  if (!(eps >= 0.f) || !(theta > 0.0) || std::isinf(theta) || std::isinf(eps)) return IVC_EINVAL;
  if (q_heads % c->kv_heads != 0 || q_heads > 65536) return IVC_EUNSUPPORTED;
  if (ld % 8 != 0 ||
      ld < (static_cast<long long>(q_heads) + 2 * c->kv_heads) * c->head_dim)
    return IVC_EUNSUPPORTED;
  if (!offsets || !q_gamma || !k_gamma || (N > 0 && (!qkv || !positions || !q_out)))
    return IVC_EINVAL;
  auto al = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  if (!al(qkv) || !al(q_gamma) || !al(k_gamma) || !al(q_out)) return IVC_EALIGN;
  if (const int rc = step_ws_ok(workspace, ws_bytes, IVC_STEP_WORKSPACE_BYTES)) return rc;
  if (N == 0 || B == 0) return IVC_OK;
  RopeFreq f = {};
  for (int j = 0; j < c->head_dim / 2; ++j)
    f.turn[j] = std::pow(theta, -2.0 * j / c->head_dim) / 6.283185307179586476925;
  const QkArgs a{static_cast<const bf16*>(qkv), ld, N, q_heads, layer, B,
                 static_cast<const bf16*>(q_gamma), static_cast<const bf16*>(k_gamma), eps,
                 positions, offsets, seqs, static_cast<bf16*>(q_out),
                 static_cast<int*>(workspace)};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  TraceScope ts("qk_norm_rope", s);
  return launch_k(c->head_dim == 64 ? qk_norm_rope_kernel<64> : qk_norm_rope_kernel<128>, dim3(N),
                  dim3(QR_THREADS), 0, s, 1, *c, a, f);
}
