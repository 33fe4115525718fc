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
// Bound by HBM (each value is read and written once). Warps work alone: a warp
// takes a token's heads, or every split-th batch of them where there are few
// tokens. D/8 lanes per head; a lane holds 4 values of the head's first half and
// the 4 of the second half that they are rotated with, so only the sum of squares
// needs shuffles (with 8 neighbouring values per lane the other halves' values
// came by shuffle, and instructions rather than HBM were the bound: 74.4 us for
// 14000 tokens of 48 heads of 128). The loads of the first batch are in flight
// while the warp finds the token's sequence, page and angles.
#include <cuda_runtime.h>

#include <cmath>

#include "ivc_internal.h"
#include "ivc_ptx.cuh"

namespace ivc {
namespace {

constexpr int QR_THREADS = 128;
constexpr int QR_WARPS = QR_THREADS / 32;
constexpr int QR_LOADS = 4;  // heads of a batch, per lane

struct RopeFreq {
  double turn[64];  // f_j / (2 pi)
};

struct QkArgs {
  const bf16* qkv;
  long long ld;
  int N, q_heads, layer, B, split;  // split: warps of a token
  const bf16* gamma_q;
  const bf16* gamma_k;
  float eps;
  const int32_t* positions;
  const int32_t* offsets;
  const int32_t* seqs;
  bf16* q_out;
  int* status;
};

__device__ __forceinline__ void unpack4(const uint2& u, float (&f)[4]) {
  f[0] = __uint_as_float(u.x << 16);
  f[1] = __uint_as_float(u.x & 0xffff0000u);
  f[2] = __uint_as_float(u.y << 16);
  f[3] = __uint_as_float(u.y & 0xffff0000u);
}
__device__ __forceinline__ uint2 pack4(const float (&f)[4]) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ uint2 load4(const bf16* p) { return *reinterpret_cast<const uint2*>(p); }
__device__ __forceinline__ void store4(bf16* p, const uint2& u) { *reinterpret_cast<uint2*>(p) = u; }

// The sequence that row tok belongs to: the last one that starts at or before it
// (0 where none does). Each step looks at 32 starts at once.
__device__ __forceinline__ int seq_of_row(const int32_t* offsets, int B, int tok, int lane) {
  int lo = 0, n = B;  // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int at = lane * step;
    const bool starts = at < n && offsets[lo + at] <= tok;
    const unsigned got = __ballot_sync(0xffffffffu, starts);
    const int last = got ? 31 - __clz(got) : 0;
    lo += last * step;
    n = min(step, n - last * step);
  }
  return lo;
}

template <int D>
__global__ void __launch_bounds__(QR_THREADS, 8)
    qk_norm_rope_kernel(const __grid_constant__ ivc_cache c, const __grid_constant__ QkArgs a,
                        const __grid_constant__ RopeFreq freq) {
  constexpr int LANES = D / 8;               // lanes per head
  constexpr int HEADS = 32 / LANES;          // heads of one load of the warp
  constexpr int BATCH = HEADS * QR_LOADS;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int unit = blockIdx.x * QR_WARPS + (threadIdx.x >> 5);
  const int tok = unit / a.split, part = unit % a.split;
  if (blockIdx.x == 0) {
    for (int b = threadIdx.x; b < a.B; b += QR_THREADS)
      if (a.offsets[b + 1] < a.offsets[b] || a.offsets[b + 1] > a.N) atomicOr(a.status, DEV_BAD_TREE);
    if (threadIdx.x == 0 && a.offsets[0] != 0) atomicOr(a.status, DEV_BAD_TREE);
  }
  if (tok >= a.N) return;
  const int heads = a.q_heads + 2 * c.kv_heads;
  const int j0 = lane % LANES * 4;           // values j0 .. j0 + 3 of both halves
  const bf16* src = a.qkv + static_cast<long long>(tok) * a.ld + j0;
  const int step = a.split * BATCH;
  int h0 = part * BATCH + lane / LANES;      // this lane's head of the batch's first load
  uint2 lo[QR_LOADS], hi[QR_LOADS];
  auto fetch = [&](int h) {
#pragma unroll
    for (int k = 0; k < QR_LOADS; ++k) {
      lo[k] = hi[k] = make_uint2(0u, 0u);
      if (h + k * HEADS < heads) {
        lo[k] = load4(src + static_cast<long long>(h + k * HEADS) * D);
        hi[k] = load4(src + static_cast<long long>(h + k * HEADS) * D + D / 2);
      }
    }
  };
  fetch(h0);
  const int end = a.offsets[a.B];
  const int pos = a.positions[tok];
  const uint2 gq0 = load4(a.gamma_q + j0), gq1 = load4(a.gamma_q + j0 + D / 2);
  const uint2 gk0 = load4(a.gamma_k + j0), gk1 = load4(a.gamma_k + j0 + D / 2);
  if (tok >= end) return;                    // behind the last sequence
  // where the token's key and value go: the first value in its page, or -1
  long long row = -1;
  {
    const int b = seq_of_row(a.offsets, a.B, tok, lane);
    const int first = a.offsets[b], s = a.seqs ? a.seqs[b] : b;
    if (s >= 0 && s < c.max_seqs && first <= tok) {
      const long long at = static_cast<long long>(c.length[s]) + tok - first;
      const int np = min(c.n_pages[s], c.max_pages);
      if (at >= 0 && at < static_cast<long long>(np) * c.page_tokens) {
        const int page = c.table[static_cast<size_t>(s) * c.max_pages + at / c.page_tokens];
        if (page >= 0 && page < c.pages)
          row = ((static_cast<long long>(a.layer) * c.pages + page) * c.kv_heads * c.page_tokens +
                 at % c.page_tokens) * D;
      }
    }
    if (row < 0 && lane == 0) atomicOr(a.status, DEV_BAD_CACHE);
  }
  // angles: lane l reduces those of D/64 rotations, a lane needs 4
  float cs[4], sn[4];
  {
    constexpr int PER = D / 64;
    float myc[PER], mys[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      double t = pos * freq.turn[lane * PER + i];
      t -= rint(t);
      sincospif(static_cast<float>(2.0 * t), &mys[i], &myc[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      cs[i] = __shfl_sync(0xffffffffu, myc[i % PER], (j0 + i) / PER);
      sn[i] = __shfl_sync(0xffffffffu, mys[i % PER], (j0 + i) / PER);
    }
  }
  const long long head_stride = static_cast<long long>(c.page_tokens) * D;
  const int normed = a.q_heads + c.kv_heads;
  const int warp_heads = (heads + HEADS - 1) / HEADS * HEADS;  // the same trips for every lane
  for (; h0 < warp_heads; h0 += step) {
#pragma unroll
    for (int k = 0; k < QR_LOADS; ++k) {
      const int h = h0 + k * HEADS;
      const bool is_q = h < a.q_heads;
      uint2 y0 = lo[k], y1 = hi[k];
      if (h - lane / LANES < normed) {  // the warp holds a q or k head
        float x0[4], x1[4], g0[4], g1[4];
        unpack4(y0, x0);
        unpack4(y1, x1);
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) ss += x0[i] * x0[i] + x1[i] * x1[i];
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float r = rsqrtf(ss * (1.f / D) + a.eps);
        unpack4(is_q ? gq0 : gk0, g0);
        unpack4(is_q ? gq1 : gk1, g1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float u = x0[i] * r * g0[i], w = x1[i] * r * g1[i];
          x0[i] = u * cs[i] - w * sn[i];
          x1[i] = w * cs[i] + u * sn[i];
        }
        if (h < normed) {
          y0 = pack4(x0);
          y1 = pack4(x1);
        }
      }
      if (h >= heads) continue;
      bf16* to = a.q_out + (static_cast<long long>(tok) * a.q_heads + h) * D + j0;
      if (!is_q) {
        if (row < 0) continue;
        to = static_cast<bf16*>(h < normed ? c.k : c.v) + row +
             (h < normed ? h - a.q_heads : h - normed) * head_stride + j0;
      }
      store4(to, y0);
      store4(to + D / 2, y1);
    }
    if (h0 + step < warp_heads) fetch(h0 + step);
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
  if (q_heads % c->kv_heads != 0 || q_heads > 65536 || N > (1 << 28)) return IVC_EUNSUPPORTED;
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
  const double ratio = std::pow(theta, -2.0 / c->head_dim);
  for (int j = 0; j < c->head_dim / 2; ++j)  // at most seven products from a power
    f.turn[j] = j % 8 ? f.turn[j - 1] * ratio
                      : std::pow(theta, -2.0 * j / c->head_dim) / 6.283185307179586476925;
  // a warp per token, or as many as the token has batches while the tokens alone
  // do not fill the SMs' warps
  const int batch = 32 / (c->head_dim / 8) * QR_LOADS;
  const int batches = (q_heads + 2 * c->kv_heads + batch - 1) / batch;
  int split = 16 * num_sms() / N;
  split = split < 1 ? 1 : split > batches ? batches : split;
  const long long blocks = (static_cast<long long>(N) * split + QR_WARPS - 1) / QR_WARPS;
  const QkArgs a{static_cast<const bf16*>(qkv), ld, N, q_heads, layer, B, split,
                 static_cast<const bf16*>(q_gamma), static_cast<const bf16*>(k_gamma), eps,
                 positions, offsets, seqs, static_cast<bf16*>(q_out),
                 static_cast<int*>(workspace)};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  TraceScope ts("qk_norm_rope", s);
  return launch_k(c->head_dim == 64 ? qk_norm_rope_kernel<64> : qk_norm_rope_kernel<128>,
                  dim3(static_cast<unsigned>(blocks)),
                  dim3(QR_THREADS), 0, s, 1, *c, a, f);
}
