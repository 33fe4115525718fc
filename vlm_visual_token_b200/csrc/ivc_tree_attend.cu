// ivc_tree_attend.cu — attention of drafted trees over the paged cache, on the
// 5th-generation tensor cores.
//
// out_i = sum_j softmax_j(scale q_i . k_j) v_j over the committed tokens, the
// node's ancestors and the node itself. One pass with the running maximum m and
// sum l: per tile of 64 keys p = e^(s - m), l = sum p, o = sum p v, all rescaled
// by e^(m - m') when the maximum rises to m'; out = o / l.
//
// What bounds it: a (sequence, kv head)'s keys and values are read from HBM once
// for up to 256 query rows (node x query head of the group), 4 D bytes a key
// against 4 D operations a row and key, so the read is the bound up to about 250
// rows, and the shape of the kernel follows the read:
//   - every CTA (one per SM, persistent) takes the same number of key tiles, a
//     contiguous piece of the list of all (sequence, row block, kv head, tile):
//     long and short sequences are cut wherever the pieces end, and the parts of
//     a cut item are merged by a second kernel in part order;
//   - keys and values come by TMA, one box per page and 64 values, into rings of
//     80 KB each;
//   - two groups of four softmax warps keep the tensor core and the exponential
//     unit busy at the same time: with more than 128 query rows each group has
//     128 rows and every tile; with fewer (plain decoding) both have the same
//     rows and every other tile, and the groups' results are merged at the end.
// Per group and tile: S[128 rows x 64 keys] = Q K^T (M 128, N 64), S read from
// TMEM (thread = row), p written back over S as bf16 and used as the A operand of
// O[128 x D] += P V (V read MN-major). A group has two S buffers, so that the
// scores of its next tile are made while it works on this one: with one buffer of
// 128 keys the scores had to wait for the weighted sum (P lies in S), each group
// idled half of the time, and 64 nodes x 4 sequences of up to 40800 tokens took
// 237 us. O stays in TMEM; it is rescaled only when a row's maximum rose by more
// than 2^8 (p then reaches 2^8 at most, which bf16 and the fp32 sums hold as
// exactly as values below 1).
//
// 48 sequences of up to 4500 tokens, one node: 153 us (705 MB, 4.6 TB/s); 24 of up to
// 6000 with 27 nodes: 133 us; 4 of up to 40800 with 64 nodes: 236 us, there bound by the
// MMAs (N = 64 takes as long as N = 128), not by HBM. These are calls on changing inputs
// one after the other for half a second, under the power cap; the first milliseconds of
// such a loop run at 137, 122 and 201 us.
//
// Registers: 168 a thread, the same for all roles (384 threads of 65536), which is less
// than the softmax warps would use: with heads of 128 they spill 256 bytes (76 with
// heads of 64).
//
// Rounding: p to bf16 for the product with v (the sum l takes the unrounded p);
// everything else is fp32 until the output. An MMA takes p in v's type; p as the sum of
// two bf16 numbers would double the MMAs of the weighted sum. The rounding costs: 0.0023
// from 64 bits (2-norm, relative) where rounding the output alone gives 0.0017.
//
// What a node does not see has no influence: unseen scores become -inf by
// selection, and in tiles that reach behind the committed tokens one warp first
// clears value rows behind the sequence and replaces non-finite values of drafted
// tokens by 0 in shared memory (0 x inf would reach every row); rows that do see
// such a token get the non-finite value back in the epilogue.
//
// Warps 0-3 and 4-7 are the softmax groups, warp 8 loads queries and keys, warp 11
// values, warps 9 and 10 issue the MMAs of one group each (and mend value tiles).
// Two of each kind, because an MMA's issue takes as long as the MMA, a barrier wait
// 150 to 350 cycles even when it is over and a load about 500: one warp's steps
// would add up to more than the 1400 cycles in which HBM delivers a tile of 32 KB
// to each SM. Every wait is bounded (IVC_DEV_WAIT_TIMEOUT).
#include <cuda.h>
#include <cuda_runtime.h>

#include "ivc_internal.h"
#include "ivc_ptx.cuh"

namespace ivc {
namespace {

constexpr int TA_THREADS = 384;
constexpr int TA_KEYS = 64;                  // keys of a tile
constexpr int TA_ROWS = 128;                 // query rows of a group
constexpr uint32_t TA_QHALF = 128 * 128;     // 128 query rows x 64 values
constexpr uint32_t TA_HALF = TA_KEYS * 128;  // a tile's keys x 64 values
constexpr int TA_MAX_BATCH = 4096;
constexpr int TA_MAX_GRID = 256;              // CTAs, one per SM
constexpr float TA_RISE = 8.f;               // log2 of the rise of m that rescales

struct TreeArgs {
  int N, q_heads, group, npt;                // npt: nodes of a 128-row tile
  int layer, B;
  float scale_log2;                          // scale * log2(e)
  const int32_t* parents;
  const int32_t* offsets;
  const int32_t* seqs;
  bf16* out;
  int* status;
  // plan, in the workspace
  long long* prefix;                         // [B + 1] tiles before sequence b
  int4* info;                                // [B] {first row, nodes, committed, sequence}
  int* start;                                // [grid] sequence in which a CTA's piece begins
  int4* head;                                // [2 grid] an item begun and not ended by a CTA
  float2* part_ml;                           // [2 grid][256] maximum (log2 units) and sum
  float4* part_o;                            // [2 grid][D / 4][256] sums, 4 values of a row
};

// The tiles are cut into as many pieces as there are CTAs, or tiles if those are
// fewer: piece i is tiles [total i / pieces, total (i + 1) / pieces), never empty.
// (Pieces of at least 4 tiles, for fewer parts to merge, measured slower: 19.2
// against 14.2 us for one sequence of 334 tokens, the same elsewhere.)
__device__ __forceinline__ int pieces_of(long long total, int grid) {
  return total < grid ? static_cast<int>(total) : grid;
}

__device__ __forceinline__ int div_up(int a, int b) { return (a + b - 1) / b; }

// ------------------------------------------------------------------ plan
// Sequence b as {first row, nodes, committed tokens, sequence}, all 0 where there
// is nothing to do, and the DEV_* bits of what is wrong with it.
__device__ __forceinline__ int4 seq_info(const ivc_cache& c, const TreeArgs& a, int b, int& bad) {
  // (all loads at once: a kernel's first tile waits for them)
  const int row = a.offsets[b], n = a.offsets[b + 1] - row;
  const int s = a.seqs ? a.seqs[b] : b;
  const bool in = s >= 0 && s < c.max_seqs;
  const int len = in ? c.length[s] : -1, np = in ? c.n_pages[s] : 0;
  const int4 none = make_int4(0, 0, 0, 0);
  if (b == 0 && row != 0) bad |= DEV_BAD_TREE;
  if (row < 0 || n < 0 || n > IVC_MAX_TREE || row > a.N - n) {
    bad |= DEV_BAD_TREE;
    return none;
  }
  if (n == 0) return none;
  if (len < 0 || np > c.max_pages ||
      static_cast<long long>(len) + n > static_cast<long long>(np) * c.page_tokens) {
    bad |= DEV_BAD_CACHE;
    return none;
  }
  return make_int4(row, n, len, s);
}
__device__ __forceinline__ long long tiles_of(const ivc_cache& c, const TreeArgs& a, const int4& info) {
  return static_cast<long long>(div_up(info.z + info.y, TA_KEYS)) * c.kv_heads *
         div_up(info.y, 2 * a.npt);
}

// One CTA: which tiles there are, and the sequence in which each piece begins.
// (Batches of up to 32 sequences do without this kernel: see Walk.)
__global__ void __launch_bounds__(1024)
    tree_plan_kernel(const __grid_constant__ ivc_cache c, const __grid_constant__ TreeArgs a,
                     int grid) {
  __shared__ long long s_prefix[TA_MAX_BATCH + 1];
  __shared__ long long s_warp[32];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = div_up(a.B, 1024);
  const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  long long mine = 0;
  int bad = 0;
  for (int b = b0; b < b1; ++b) {
    const int4 info = seq_info(c, a, b, bad);
    a.info[b] = info;
    s_prefix[b] = mine;  // within the thread; completed below
    mine += tiles_of(c, a, info);
  }
  if (bad) atomicOr(a.status, bad);
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  long long before = incl - mine;
  for (int w = 0; w < warp; ++w) before += s_warp[w];
  for (int b = b0; b < b1; ++b) {
    s_prefix[b] += before;
    a.prefix[b] = s_prefix[b];
  }
  if (tid == 1023) {
    s_prefix[a.B] = before + mine;
    a.prefix[a.B] = before + mine;
  }
  __syncthreads();
  const long long total = s_prefix[a.B];
  const int pieces = pieces_of(total, grid);
  for (int i = tid; i < grid; i += 1024) {
    if (i >= pieces) continue;
    const long long pos = total * i / pieces;  // the last sequence that begins at or before it
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_prefix[mid] <= pos) lo = mid; else hi = mid;
    }
    a.start[i] = lo;
  }
}

// ------------------------------------------------------------------ items
// A CTA's part of one (sequence, block of up to 2 npt nodes, kv head).
struct Item {
  int row, n, len, seq;   // of the sequence: first row, nodes, committed tokens
  int h;                  // kv head
  int node0, nodes;       // of the block
  int t0, t1;             // key tiles of this part
  bool rows2;             // more than 128 rows: each group has its own
  bool begins, ends;      // the part holds the item's first / last tile
  __device__ int units() const { return rows2 ? 2 * (t1 - t0) : t1 - t0; }
};

// Walks a CTA's piece; every role of the CTA walks it for itself. Only the first
// item is found by division; the ones after it are the next head, block of nodes
// or sequence, whose info is read one sequence ahead.
//
// A batch of up to 32 sequences is planned by each warp for itself, lane b holding
// sequence b: a kernel less in the stream (4 of 14 us for one short sequence).
struct Walk {
  long long left;         // tiles of the piece not walked yet
  long long total;        // of all pieces
  int b, q, t0;           // sequence, item of the sequence (block * kv_heads + head), tile
  int4 info, ahead;       // of sequences b and b + 1
  int4 lane_info;         // of sequence `lane`, small batches
  __device__ int4 info_of(const TreeArgs& a, int s) const {
    if (a.B > 32) return s < a.B ? a.info[s] : make_int4(0, 0, 0, 0);
    const unsigned all = 0xffffffffu;  // lanes behind the batch hold 0
    return s < 32 ? make_int4(__shfl_sync(all, lane_info.x, s), __shfl_sync(all, lane_info.y, s),
                              __shfl_sync(all, lane_info.z, s), __shfl_sync(all, lane_info.w, s))
                  : make_int4(0, 0, 0, 0);
  }
  // By a whole warp, as next() is. `status`: null but in one warp of the grid.
  __device__ Walk(const ivc_cache& c, const TreeArgs& a, int* status) {
    const int i = blockIdx.x;
    long long pos = 0, first = 0;
    lane_info = make_int4(0, 0, 0, 0);
    left = 0;
    if (a.B > 32) {
      total = a.prefix[a.B];
    } else {
      const int lane = threadIdx.x & 31;
      int bad = 0;
      if (lane < a.B) lane_info = seq_info(c, a, lane, bad);
      if (bad && status != nullptr) atomicOr(status, bad);
      const long long mine = tiles_of(c, a, lane_info);
      long long incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      total = __shfl_sync(0xffffffffu, incl, 31);
      const int pieces = pieces_of(total, gridDim.x);
      if (i < pieces) pos = total * i / pieces;
      b = min(31, __popc(__ballot_sync(0xffffffffu, incl <= pos)));  // the first that ends behind it
      first = __shfl_sync(0xffffffffu, incl - mine, b);
    }
    const int pieces = pieces_of(total, gridDim.x);
    if (i >= pieces) return;
    if (a.B > 32) {
      pos = total * i / pieces;
      b = a.start[i];
      first = a.prefix[b];
    }
    left = total * (i + 1) / pieces - pos;
    info = info_of(a, b);
    ahead = info_of(a, b + 1);
    const int tiles = div_up(info.z + info.y, TA_KEYS);
    q = static_cast<int>((pos - first) / tiles);
    t0 = static_cast<int>((pos - first) % tiles);
  }
  __device__ bool next(const ivc_cache& c, const TreeArgs& a, Item& it) {
    if (left <= 0) return false;
    while (info.y == 0 || q == c.kv_heads * div_up(info.y, 2 * a.npt)) {
      ++b;  // there are tiles left, so there is a sequence with nodes
      info = ahead;
      ahead = info_of(a, b + 1);
      q = 0;
    }
    it.row = info.x;
    it.n = info.y;
    it.len = info.z;
    it.seq = info.w;
    const int tiles = div_up(it.len + it.n, TA_KEYS);
    it.t0 = t0;
    it.t1 = static_cast<int>(min(static_cast<long long>(tiles), t0 + left));
    const int block = q / c.kv_heads;
    it.h = q - block * c.kv_heads;
    it.node0 = block * 2 * a.npt;
    it.nodes = min(2 * a.npt, it.n - it.node0);
    it.rows2 = it.nodes > a.npt;
    it.begins = it.t0 == 0;
    it.ends = it.t1 == tiles;
    left -= it.t1 - it.t0;
    ++q;
    t0 = 0;
    return true;
  }
};

// ------------------------------------------------------------------ tcgen05 pieces
// A bounded wait of a whole warp: every lane gets the same answer.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}
// Whether the phase is over, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return done != 0;
}
// One lane of a converged warp, always the same. The compiler knows that a branch
// on it is taken by one lane, which a branch on the lane number hides from it.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}
// D[tmem] (+)= A[tmem, bf16 pairs] * B[smem desc].
__device__ __forceinline__ void umma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                             uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

template <int D>
struct TaSmem {
  static constexpr int HALVES = D / 64;
  static constexpr uint32_t SLOT = HALVES * TA_HALF;    // one tile of keys or values
  static constexpr int SLOTS = 81920 / SLOT;            // of keys, and of values: 80 KB each
  static constexpr uint32_t Q = 2 * HALVES * TA_QHALF;  // two groups' rows
  static constexpr uint32_t TOTAL = 1024 + Q + 2 * SLOTS * SLOT;
};

// The keys that a node sees in the tile at t0 as bits: committed tokens, and
// behind them the node's ancestors and itself (anc).
__device__ __forceinline__ void tile_mask(const uint32_t (&anc)[4], int len, int t0,
                                          uint32_t (&mask)[2]) {
  const int shift = len - t0;  // tile position of node 0
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const int below = shift - 32 * w;  // committed tokens in this word
    uint32_t m = below >= 32 ? 0xffffffffu : below <= 0 ? 0u : (1u << below) - 1u;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int s = below + 32 * x;  // anc word x starts at bit s of this word
      if (s > -32 && s < 32) m |= s >= 0 ? anc[x] << s : anc[x] >> -s;
    }
    mask[w] = m;
  }
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Value rows of the tile at `base` behind the committed tokens: those of drafted
// tokens lose their non-finite values (and *odd tells so), those behind the
// sequence become 0 up to the end of its last page (further ones were loaded as 0).
// By one warp, in 16-byte pieces; the swizzle only permutes pieces within a row.
template <int D>
__device__ void mend_values(uint8_t* v, int base, int len, int n, int page_tokens, int* odd, int lane) {
  const int drafted = max(0, len - base), behind = min(TA_KEYS, len + n - base);
  const int end = min(TA_KEYS, div_up(len + n, page_tokens) * page_tokens - base);
  constexpr int HALVES = D / 64, BATCH = 4;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  auto piece = [&](int i, int hf) {
    return reinterpret_cast<uint4*>(v + hf * TA_HALF + (i >> 3) * 128 + (i & 7) * 16);
  };
  for (int i = behind * 8 + lane; i < end * 8; i += 32)
#pragma unroll
    for (int hf = 0; hf < HALVES; ++hf) *piece(i, hf) = zero;
  bool found = false;
  for (int i0 = drafted * 8 + lane; i0 < behind * 8; i0 += 32 * BATCH) {
    uint4 x[BATCH][HALVES];  // all loads of a batch before the first test
#pragma unroll
    for (int k = 0; k < BATCH; ++k)
#pragma unroll
      for (int hf = 0; hf < HALVES; ++hf)
        x[k][hf] = i0 + 32 * k < behind * 8 ? *piece(i0 + 32 * k, hf) : zero;
#pragma unroll
    for (int k = 0; k < BATCH; ++k)
#pragma unroll
      for (int hf = 0; hf < HALVES; ++hf) {
        uint32_t w[4] = {x[k][hf].x, x[k][hf].y, x[k][hf].z, x[k][hf].w};
        bool here = false;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if ((w[j] & 0x7f80u) == 0x7f80u) { w[j] &= 0xffff0000u; here = true; }
          if ((w[j] & 0x7f800000u) == 0x7f800000u) { w[j] &= 0x0000ffffu; here = true; }
        }
        if (here) {
          *piece(i0 + 32 * k, hf) = make_uint4(w[0], w[1], w[2], w[3]);
          found = true;
        }
      }
  }
  if (found) *odd = 1;
  __threadfence_block();  // the flag is read behind a barrier that a tcgen05.commit completes
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
}

template <int D>
__global__ void __launch_bounds__(TA_THREADS, 1)
    tree_attend_kernel(const __grid_constant__ CUtensorMap qmap,
                       const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap,
                       const __grid_constant__ ivc_cache c, const __grid_constant__ TreeArgs a) {
  using S = TaSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sq = sm;
  uint8_t* kring = sm + S::Q;
  uint8_t* vring = kring + S::SLOTS * S::SLOT;
  __shared__ __align__(8) uint64_t kfull[S::SLOTS], kempty[S::SLOTS];
  __shared__ __align__(8) uint64_t vfull[S::SLOTS], vempty[S::SLOTS];
  __shared__ __align__(8) uint64_t qfull[2], qempty[2];  // of each 128-row buffer
  __shared__ __align__(8) uint64_t sfull[2][2], pready[2][2], odone[2];  // [group][S buffer]
  __shared__ __align__(8) uint64_t ofull, ofree, mlready, mended, seen, drained[2];
  __shared__ uint32_t s_tmem;
  __shared__ int s_odd[2][2];       // [item & 1][issuer]: a drafted value is not finite
  __shared__ float2 s_ml[TA_ROWS];  // group 1's maximum and sum
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::SLOTS; ++s) {
      mbar_init(&kfull[s], 1);
      mbar_init(&kempty[s], 2);  // both issuers
      mbar_init(&vfull[s], 1);
      mbar_init(&vempty[s], 2);
    }
    for (int g = 0; g < 2; ++g) {
      for (int buf = 0; buf < 2; ++buf) {
        mbar_init(&sfull[g][buf], 1);
        mbar_init(&pready[g][buf], 4);
      }
      mbar_init(&odone[g], 1);
      mbar_init(&drained[g], 1);
      mbar_init(&qfull[g], 1);
      mbar_init(&qempty[g], 2);
    }
    mbar_init(&ofull, 2);
    mbar_init(&ofree, 8);
    mbar_init(&mlready, 4);
    mbar_init(&mended, 1);
    mbar_init(&seen, 1);
    fence_mbar_init();
    tma_prefetch_desc(&qmap);
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
  }
  if (warp == 9) {
    tmem_alloc(&s_tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // all 512 columns were asked for, so the base is 0; as a constant it spares the
  // MMAs a register each
  constexpr uint32_t tmem = 0;
  bool ok = true;
  pdl_wait();     // the plan; everything before it in the stream
  pdl_trigger();  // the merge may launch; it waits for this grid

  if (warp == 8 || warp == 11) {
    // ------------------------------------------------------------- producers
    const bool keys = warp == 8;
    const CUtensorMap* map = keys ? &kmap : &vmap;
    uint8_t* ring = keys ? kring : vring;
    uint64_t* full = keys ? kfull : vfull;
    uint64_t* empty = keys ? kempty : vempty;
    const int pt = c.page_tokens, box = min(pt, TA_KEYS), per_tile = TA_KEYS / box;
    const int pt_log = 31 - __clz(pt), box_log = 31 - __clz(box);
    const int nowhere = c.pages * c.kv_heads * pt;  // behind the last row: reads as 0
    Walk walk(c, a, keys && blockIdx.x == 0 ? a.status : nullptr);
    Item it = {};
    int slot = 0, round = 0, queries = 0;
    // rows of the boxes (a page or half of one) of an item: lane l holds those of
    // boxes base + l and base + 32 + l, so that the table is read 32 boxes ahead
    auto row_of = [&](int b) -> int {
      const int token = b << box_log;
      if (token >= it.len + it.n) return nowhere;
      const int page = c.table[static_cast<size_t>(it.seq) * c.max_pages + (token >> pt_log)];
      if (page < 0 || page >= c.pages) {
        atomicOr(a.status, DEV_BAD_CACHE);
        return nowhere;
      }
      return (page * c.kv_heads + it.h) * pt + (token & (pt - 1));
    };
    // a 128-row buffer of queries, in turn
    auto load_q = [&](int node0) {
      const int buf = queries & 1;
      if (!warp_wait(&qempty[buf], ((queries >> 1) & 1) ^ 1)) return false;
      ++queries;
      if (elect_one()) {
        mbar_arrive_expect_tx(&qfull[buf], S::HALVES * a.npt * a.group * 128);
#pragma unroll
        for (int hf = 0; hf < S::HALVES; ++hf)
          tma_load_3d(sq + (buf * S::HALVES + hf) * TA_QHALF, &qmap, &qfull[buf], 64 * hf,
                      it.h * a.group, node0);
      }
      __syncwarp();
      return true;
    };
    while (ok && walk.next(c, a, it)) {
      if (keys) ok = load_q(it.row + it.node0);
      if (ok && keys && it.rows2) ok = load_q(it.row + it.node0 + a.npt);
      int base = it.t0 * per_tile & ~31;
      int now = row_of(base + lane), next = row_of(base + 32 + lane);
      for (int tile = it.t0; tile < it.t1 && ok; ++tile) {
        const int first = tile * per_tile;
        if (first >= base + 32) {
          base += 32;
          now = next;
          next = row_of(base + 32 + lane);
        }
        int row[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) row[i] = __shfl_sync(0xffffffffu, now, (first + i) & 31);
        ok = warp_wait(&empty[slot], (round & 1) ^ 1);
        if (!ok) break;
        if (elect_one()) {
          uint8_t* dst = ring + slot * S::SLOT;
          mbar_arrive_expect_tx(&full[slot], S::SLOT);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i < per_tile)
#pragma unroll
              for (int hf = 0; hf < S::HALVES; ++hf)
                tma_load_2d(dst + hf * TA_HALF + i * box * 128, map, &full[slot], 64 * hf, row[i]);
        }
        __syncwarp();
        if (++slot == S::SLOTS) {
          slot = 0;
          ++round;
        }
      }
      // a single node has no parent to walk to; whether it names one is looked up here
      if (!keys && it.n == 1 && it.h == 0 && it.begins && lane == 0 && a.parents != nullptr &&
          a.parents[it.row] != -1)
        atomicOr(a.status, DEV_BAD_TREE);
    }
    if (!ok) {  // let the copies in flight land
      const int loads = round * S::SLOTS + slot;
      for (int i = max(0, loads - S::SLOTS); i < loads; ++i)
        mbar_wait(&full[i % S::SLOTS], (i / S::SLOTS) & 1);
      for (int i = max(0, queries - 2); i < queries; ++i) mbar_wait(&qfull[i & 1], (i >> 1) & 1);
    }
  } else if (warp == 9 || warp == 10) {
    // ------------------------------------------------------------- MMA issuers
    // unit u: group u & 1, tile u / 2 (own rows) or u (own tiles), S buffer
    // u / 2 & 1. Scores of unit u + 4 follow the weighted sum of unit u, whose
    // weights lie in the same columns. Each warp issues its group's units, but
    // takes every load in turn (a barrier's phases cannot be skipped) and, where
    // a tile is not its own, gives it back at once.
    const int g = warp - 9;
    const uint32_t idesc_s = idesc_bf16_f32(128, TA_KEYS);
    const uint32_t idesc_o = idesc_bf16_f32(128, D) | (1u << 16);  // B MN-major
    const uint64_t kdesc = sw128_kmajor_desc(smem_u32(kring));
    const uint64_t vdesc = sw128_mnmajor_desc(smem_u32(vring), TA_HALF);
    Walk walk(c, a, nullptr);
    Item it = {};
    int items = 0, mends = 0, queries = 0;
    int ks = 0, kround = 0, vs = 0, vround = 0;  // the next tile's slots
    uint32_t np = 0;                             // bit buffer: phase of the weights
    auto advance = [&](int& slot, int& round) {
      if (++slot == S::SLOTS) {
        slot = 0;
        ++round;
      }
    };
    while (ok && walk.next(c, a, it)) {
      const int U = it.units(), mine = (U + 1 - g) / 2;
      const bool all = it.rows2;           // every tile is used by both groups
      const int T = it.t1 - it.t0, ahead = all ? 2 : 4;
      auto own = [&](int t) { return all || (t & 1) == g; };
      // the queries: one buffer, or group 0's and group 1's
      const int qb = queries & 1, my_q = all ? qb ^ g : qb;
      ok = warp_wait(&qfull[qb], (queries >> 1) & 1);
      ++queries;
      if (ok && all) {
        ok = warp_wait(&qfull[queries & 1], (queries >> 1) & 1);
        ++queries;
      }
      if (!ok) break;
      const uint64_t qdesc = sw128_kmajor_desc(smem_u32(sq) + my_q * S::HALVES * TA_QHALF);
      if (all && lane == 0) mbar_arrive(&qempty[my_q ^ 1]);  // the other group's buffer
      // by one lane: this group's scores with the keys of its unit i ...
      auto issue_scores = [&](int i) {
        const uint64_t bd = kdesc + (ks * S::SLOT >> 4);
        const int buf = i & 1;
#pragma unroll
        for (int hf = 0; hf < S::HALVES; ++hf)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_bf16(tmem + 128 * g + 64 * buf, qdesc + (hf * TA_QHALF >> 4) + 2 * kk,
                      bd + (hf * TA_HALF >> 4) + 2 * kk, idesc_s, (hf | kk) != 0);
        umma_commit(&sfull[g][buf]);
        umma_commit(&kempty[ks]);
        if (i == mine - 1) umma_commit(&qempty[my_q]);
      };
      // ... and its weighted sum of the values of unit i
      auto issue_sum = [&](int i) {
        const uint64_t bd = vdesc + (vs * S::SLOT >> 4);
        const int buf = i & 1;
#pragma unroll
        for (int kk = 0; kk < TA_KEYS / 16; ++kk)
          umma_bf16_ta(tmem + 256 + 128 * g, tmem + 128 * g + 64 * buf + 8 * kk,
                       bd + ((2048 * kk) >> 4), idesc_o, (i != 0 || kk != 0) ? 1u : 0u);
        umma_commit(&odone[g]);
        umma_commit(&vempty[vs]);
        if (i == mine - 1) umma_commit(&ofull);
      };
      for (int t = 0; t < ahead && t < T && ok; ++t) {
        ok = warp_wait(&kfull[ks], kround & 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          if (own(t)) issue_scores(all ? t : t >> 1);
          else mbar_arrive(&kempty[ks]);
        }
        __syncwarp();
        advance(ks, kround);
      }
      if (ok && mine == 0) {               // a single tile: nothing for group 1, which
        ok = warp_wait(&ofree, (items & 1) ^ 1);  // must not count for the item before
        if (ok && lane == 0) {
          s_odd[items & 1][g] = 0;
          mbar_arrive(&qempty[my_q]);
          mbar_arrive(&ofull);
        }
        __syncwarp();
      }
      int done = 0;                        // own units summed
      for (int t = 0; t < T && ok; ++t) {
        const bool more = t + ahead < T, mine_now = own(t);
        const int buf = done & 1;
        // the values, the weights and the keys of the scores that follow: one wait
        // for all three, and one branch with all MMAs of the step
        long long since = 0;
        while (!__all_sync(0xffffffffu,
                           mbar_test(&vfull[vs], vround & 1) &&
                               (!more || mbar_test(&kfull[ks], kround & 1)) &&
                               (!mine_now || mbar_test(&pready[g][buf], (np >> buf) & 1)))) {
          const long long now = clock64();
          if (since == 0) since = now;
          if (__any_sync(0xffffffffu, now - since > IVC_WAIT_CYCLES)) { ok = false; break; }
        }
        if (ok && mine_now && done == 0) {
          ok = warp_wait(&ofree, (items & 1) ^ 1);
          if (lane == 0) s_odd[items & 1][g] = 0;  // no epilogue reads it any more
          __threadfence_block();
        }
        if (!ok) break;
        const int tile = it.t0 + t;
        if (mine_now && (tile + 1) * TA_KEYS > it.len) {  // reaches behind the committed tokens
          if (!all || g == 0) {
            __syncwarp();
            mend_values<D>(vring + vs * S::SLOT, tile * TA_KEYS, it.len, it.n, c.page_tokens,
                           &s_odd[items & 1][g], lane);
          }
          if (all && g == 0) {  // the other issuer, which has seen the tile before
            ok = warp_wait(&seen, (mends & 1) ^ 1);
            if (ok && lane == 0) mbar_arrive(&mended);
            ++mends;
          } else if (all) {
            ok = warp_wait(&mended, mends++ & 1);
            if (ok && lane == 0) mbar_arrive(&seen);
          }
          if (!ok) break;
        }
        tc_fence_after();
        if (elect_one()) {
          if (mine_now) {
            issue_sum(done);
            if (more) issue_scores(all ? t + ahead : (t + ahead) >> 1);
          } else {
            mbar_arrive(&vempty[vs]);
            if (more) mbar_arrive(&kempty[ks]);
          }
        }
        __syncwarp();
        if (mine_now) {
          np ^= 1u << buf;
          ++done;
        }
        advance(vs, vround);
        if (more) advance(ks, kround);
      }
      ++items;
    }
    if (!ok) {  // let the MMAs in flight end before the TMEM is given back
      if (elect_one()) umma_commit(&drained[g]);
      __syncwarp();
      warp_wait(&drained[g], 0);
    }
  } else if (warp < 8) {
    // ------------------------------------------------------ softmax, epilogue
    const int g = warp >> 2, quad = warp & 3;
    const int r = quad * 32 + lane;                   // row of the group = TMEM lane
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t to = tmem + lanes + 256 + 128 * g;
    const int first_lane_row = quad * 32;
    const int row_node = r / a.group, row_head = r - row_node * a.group;  // within a block of rows
    Walk walk(c, a, nullptr);
    Item it = {};
    if (threadIdx.x == 0) {  // for the merge
      a.head[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
      if (blockIdx.x == 0 && a.B <= 32) a.prefix[a.B] = walk.total;
    }
    int items = 0, nml = 0, sums = 0;  // sums: weighted sums asked for by this group
    uint32_t ns = 0;                   // bit buffer: phase of the scores
    while (ok && walk.next(c, a, it)) {
      const int U = it.units();
      const int node0 = it.node0 + (it.rows2 ? g * a.npt : 0);        // of the group
      const int gnodes = min(a.npt, it.node0 + it.nodes - node0);
      const int rows = gnodes * a.group;
      const bool live = first_lane_row < rows;                        // the warp has rows
      const int node = node0 + row_node;
      uint32_t anc[4] = {0u, 0u, 0u, 0u};
      if (it.n == 1) {
        anc[0] = 1u;
      } else if (live && it.t1 * TA_KEYS > it.len) {
        // parents of nodes 4 lane .. 4 lane + 3 in the bytes of one register
        uint32_t packed = 0;
        bool bad = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = 4 * lane + e;
          int par = i - 1;
          if (i < it.n && a.parents) {
            par = a.parents[it.row + i];
            if (par < -1 || par >= i) { par = -1; bad = true; }
          }
          packed |= static_cast<uint32_t>(par & 0xff) << (8 * e);
        }
        if (bad) atomicOr(a.status, DEV_BAD_TREE);
        int i = r < rows ? node : -1;
        while (__any_sync(0xffffffffu, i >= 0)) {
          const int at = max(i, 0);
#pragma unroll
          for (int w = 0; w < 4; ++w)
            if (i >= 0 && (at >> 5) == w) anc[w] |= 1u << (at & 31);
          const uint32_t four = __shfl_sync(0xffffffffu, packed, at >> 2);
          const int par = static_cast<int8_t>((four >> (8 * (at & 3))) & 0xff);
          i = i < 0 ? -1 : par;
        }
      }
      float m = -INFINITY, l = 0.f;   // the maximum that p is taken against, in log2 units
      for (int u = g; u < U && ok; u += 2) {
        const int buf = (u >> 1) & 1;
        const uint32_t ts = tmem + lanes + 128 * g + 64 * buf;
        ok = warp_wait(&sfull[g][buf], (ns >> buf) & 1);
        if (!ok) break;
        ns ^= 1u << buf;
        tc_fence_after();
        if (live) {
          const int tile = it.t0 + (it.rows2 ? u >> 1 : u);
          uint32_t x0[32], x1[32];
          tmem_ld32(ts, x0);
          tmem_ld32(ts + 32, x1);
          tmem_ld_wait();
          if ((tile + 1) * TA_KEYS > it.len) {
            uint32_t mask[2];
            tile_mask(anc, it.len, tile * TA_KEYS, mask);
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              if (!((mask[0] >> j) & 1)) x0[j] = 0xff800000u;  // -inf
              if (!((mask[1] >> j) & 1)) x1[j] = 0xff800000u;
            }
          }
          float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            t0 = max3(t0, __uint_as_float(x0[j]), __uint_as_float(x0[j + 1]));
            t1 = max3(t1, __uint_as_float(x1[j]), __uint_as_float(x1[j + 1]));
          }
          const float rise = fmaxf(t0, t1) * a.scale_log2;
          if (u < 2) {
            m = rise;
          } else if (const bool mine = r < rows && rise - m > TA_RISE; __any_sync(0xffffffffu, mine)) {
            // a row is rescaled by its own scores alone (f is 1 for the others of the
            // warp): its result does not depend on the rows beside it, nor on what
            // shared memory held in those behind the block's last one. Once this
            // group's sum before is complete (the one before that is: these scores lie
            // in the columns of its weights)
            ok = warp_wait(&odone[g], (sums - 1) & 1);
            if (!ok) break;
            tc_fence_after();
            const float f = mine ? ex2(m - rise) : 1.f;
            if (mine) m = rise;
            l *= f;
#pragma unroll
            for (int d = 0; d < D; d += 32) {
              uint32_t o[32];
              tmem_ld32(to + d, o);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              tmem_st32(to + d, o);
            }
          }
          const float base = m == -INFINITY ? 0.f : m;
          float sum0 = 0.f, sum1 = 0.f;
          uint32_t p[32];
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float e0 = ex2(fmaf(__uint_as_float(x0[j]), a.scale_log2, -base));
            const float e1 = ex2(fmaf(__uint_as_float(x0[j + 1]), a.scale_log2, -base));
            const float e2 = ex2(fmaf(__uint_as_float(x1[j]), a.scale_log2, -base));
            const float e3 = ex2(fmaf(__uint_as_float(x1[j + 1]), a.scale_log2, -base));
            sum0 += e0 + e1;
            sum1 += e2 + e3;
            p[j / 2] = pack_bf16(e0, e1);
            p[16 + j / 2] = pack_bf16(e2, e3);
          }
          tmem_st32(ts, p);
          l += sum0 + sum1;
          tmem_st_wait();
        }
        ++sums;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pready[g][buf]);
      }
      // ---------------------------------------------------------- epilogue
      const bool two = !it.rows2 && U > 1;  // both groups have sums of the same rows
      ok = ok && warp_wait(&ofull, items & 1);
      if (!ok) break;
      if (!it.rows2 && g == 1) {  // group 0 merges and writes
        if (two) {
          s_ml[r] = make_float2(m, l);
          __syncwarp();
          if (lane == 0) mbar_arrive(&mlready);
        }
        if (lane == 0) mbar_arrive(&ofree);
        ++items;
        continue;
      }
      if (two) ok = warp_wait(&mlready, nml++ & 1);
      if (!ok) break;
      tc_fence_after();
      if (live) {
        float m1 = -INFINITY, l1 = 0.f;
        if (two) {
          const float2 ml = s_ml[r];
          m1 = ml.x;
          l1 = ml.y;
        }
        const float m2 = fmaxf(m, m1);
        const float f0 = m == -INFINITY ? 0.f : ex2(m - m2);
        const float f1 = m1 == -INFINITY ? 0.f : ex2(m1 - m2);
        // (a row whose scores are NaN keeps a NaN sum)
        const float sum = (m == -INFINITY ? l : l * f0) + (m1 == -INFINITY ? l1 : l1 * f1);
        const bool whole = it.begins && it.ends;
        const float inv = whole ? 1.f / sum : 1.f;
        const bool write = r < rows;
        const int slot = 2 * blockIdx.x + (it.begins ? 1 : 0);
        const int prow = (it.rows2 ? g * TA_ROWS : 0) + r;
        bf16* dst = a.out + (static_cast<long long>(it.row + node) * a.q_heads +
                             it.h * a.group + row_head) * D;
        float4* part = a.part_o + static_cast<size_t>(slot) * (D / 4) * 256 + prow;
        const bool odd = it.t1 * TA_KEYS > it.len && (s_odd[items & 1][0] | s_odd[items & 1][1]) != 0;
#pragma unroll 1
        for (int d = 0; d < D; d += 32) {
          __syncwarp();
          uint32_t o[32];
          tmem_ld32(to + d, o);
          if (two) {
            uint32_t o1[32];
            tmem_ld32(to + 128 + d, o1);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j)
              o[j] = __float_as_uint((__uint_as_float(o[j]) * f0 + __uint_as_float(o1[j]) * f1) * inv);
          } else {
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * inv);
          }
          if (!write) continue;
          if (odd) {  // non-finite values of drafted tokens that this row sees
            for (int i = max(0, it.t0 * TA_KEYS - it.len); i < it.n; ++i) {
              const int t = it.len + i;
              if (t >= it.t1 * TA_KEYS) break;
              const uint32_t word = i < 64 ? (i < 32 ? anc[0] : anc[1]) : (i < 96 ? anc[2] : anc[3]);
              if (!((word >> (i & 31)) & 1)) continue;
              const int page = c.table[static_cast<size_t>(it.seq) * c.max_pages + t / c.page_tokens];
              if (page < 0 || page >= c.pages) continue;
              const bf16* v = static_cast<const bf16*>(c.v) +
                              (((static_cast<size_t>(a.layer) * c.pages + page) * c.kv_heads + it.h) *
                                   c.page_tokens + t % c.page_tokens) * D + d;
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                const float y = __bfloat162float(v[j]);
                if (!isfinite(y)) o[j] = __float_as_uint(__uint_as_float(o[j]) + y);
              }
            }
          }
          if (whole) {
            uint4* to16 = reinterpret_cast<uint4*>(dst + d);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t w[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                w[k] = pack_bf16(__uint_as_float(o[8 * j + 2 * k]), __uint_as_float(o[8 * j + 2 * k + 1]));
              to16[j] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)  // neighbouring lanes, neighbouring 16 bytes
              part[(d / 4 + j) * 256] =
                  make_float4(__uint_as_float(o[4 * j]), __uint_as_float(o[4 * j + 1]),
                              __uint_as_float(o[4 * j + 2]), __uint_as_float(o[4 * j + 3]));
          }
        }
        if (write && !whole)
          a.part_ml[static_cast<size_t>(slot) * 256 + prow] = make_float2(two ? m2 : m, sum);
      }
      if (g == 0 && warp == 0 && lane == 0 && it.begins && !it.ends) {
        // the merge's work: the parts that follow are those of the next CTAs
        a.head[2 * blockIdx.x] = make_int4(1, it.row, it.node0, it.nodes);
        a.head[2 * blockIdx.x + 1] =
            make_int4(it.h, it.rows2, div_up(it.len + it.n, TA_KEYS) - it.t1, 0);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ofree);
      ++items;
    }
  }
  if (!ok) atomicOr(a.status, DEV_WAIT_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(s_tmem, 512);
  }
}

// ------------------------------------------------------------------ merge
// Blocks (i, y) merge the item that CTA i began and did not end, if there is one:
// its parts are CTA i's and, in order, the first ones of the CTAs after it. A
// thread has 4 values of a row, rows fastest, and 8 parts in flight.
constexpr int TM_THREADS = 256;
constexpr int TM_PARTS = 8;
template <int D>
__global__ void __launch_bounds__(TM_THREADS)
    tree_merge_kernel(const __grid_constant__ ivc_cache c, const __grid_constant__ TreeArgs a,
                      int grid) {
  pdl_wait();
  pdl_trigger();
  const int i = blockIdx.x;
  const int4 h0 = a.head[2 * i];      // {1, first row of the sequence, first node, nodes}
  const int4 h1 = a.head[2 * i + 1];  // {kv head, more than 128 rows, tiles that follow, 0}
  if (h0.x != 1) return;
  // its parts: the pieces that begin before it ends
  const long long total = a.prefix[a.B];
  const int pieces = pieces_of(total, grid);
  const long long item_end = total * (i + 1) / pieces + h1.z;
  const int parts =
      static_cast<int>(min(static_cast<long long>(pieces), (item_end * pieces + total - 1) / total)) - i;
  auto slot = [&](int k) { return static_cast<size_t>(k == 0 ? 2 * i + 1 : 2 * (i + k)); };
  const int rows = h0.w * a.group, full = a.npt * a.group;  // live ones; of group 0
  for (int e = blockIdx.y * TM_THREADS + threadIdx.x; e < rows * (D / 4);
       e += gridDim.y * TM_THREADS) {
    const int live = e % rows, d4 = e / rows;
    const int row = live < full ? live : TA_ROWS + live - full;
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < parts; k0 += TM_PARTS) {
      float2 ml[TM_PARTS];
      float4 x[TM_PARTS];
#pragma unroll
      for (int k = 0; k < TM_PARTS; ++k) {
        ml[k] = make_float2(-INFINITY, 0.f);
        x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k0 + k < parts) {
          ml[k] = a.part_ml[slot(k0 + k) * 256 + row];
          x[k] = a.part_o[(slot(k0 + k) * (D / 4) + d4) * 256 + row];
        }
      }
      float top = m;
#pragma unroll
      for (int k = 0; k < TM_PARTS; ++k) top = fmaxf(top, ml[k].x);
      const float f0 = m == -INFINITY ? 1.f : ex2(m - top);
      m = top;
      l *= f0;
      o = make_float4(o.x * f0, o.y * f0, o.z * f0, o.w * f0);
#pragma unroll
      for (int k = 0; k < TM_PARTS; ++k) {
        if (ml[k].x == -INFINITY && ml[k].y == 0.f) continue;  // it saw nothing in that part
        const float f = ml[k].x == -INFINITY ? 1.f : ex2(ml[k].x - top);
        l += ml[k].y * f;
        o.x += x[k].x * f;
        o.y += x[k].y * f;
        o.z += x[k].z * f;
        o.w += x[k].w * f;
      }
    }
    const float inv = 1.f / l;
    bf16* dst = a.out + (static_cast<long long>(h0.y + h0.z + live / a.group) * a.q_heads +
                         h1.x * a.group + live % a.group) * D + 4 * d4;
    *reinterpret_cast<uint2*>(dst) =
        make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
  }
}

int tree_grid() { return num_sms() < TA_MAX_GRID ? num_sms() : TA_MAX_GRID; }

size_t up256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

// Places the plan and the parts behind the status word; the bytes needed.
size_t carve(TreeArgs* a, char* ws, int B, int grid, int D) {
  size_t at = 256;
  auto take = [&](size_t bytes) {
    char* p = ws ? ws + at : nullptr;
    at += up256(bytes);
    return p;
  };
  char* prefix = take(static_cast<size_t>(B + 1) * 8);
  char* info = take(static_cast<size_t>(B) * 16);
  char* start = take(static_cast<size_t>(grid) * 4);
  char* head = take(static_cast<size_t>(grid) * 32);
  char* ml = take(static_cast<size_t>(grid) * 2 * 256 * 8);
  char* o = take(static_cast<size_t>(grid) * 2 * 256 * D * 4);
  if (a) {
    a->prefix = reinterpret_cast<long long*>(prefix);
    a->info = reinterpret_cast<int4*>(info);
    a->start = reinterpret_cast<int*>(start);
    a->head = reinterpret_cast<int4*>(head);
    a->part_ml = reinterpret_cast<float2*>(ml);
    a->part_o = reinterpret_cast<float4*>(o);
  }
  return at;
}

template <int D>
int run_tree(const CUtensorMap& qm, const CUtensorMap& km, const CUtensorMap& vm,
             const ivc_cache& c, const TreeArgs& a, int grid, cudaStream_t s) {
  const void* kern = reinterpret_cast<const void*>(tree_attend_kernel<D>);
  if (const int rc = smem_optin(kern, TaSmem<D>::TOTAL)) return rc;
  if (a.B > 32) {
    TraceScope ts("tree.plan", s);
    if (const int rc = launch_k(tree_plan_kernel, dim3(1), dim3(1024), 0, s, 1, c, a, grid)) return rc;
  }
  {
    TraceScope ts("tree.attend", s);
    if (const int rc = launch_k(tree_attend_kernel<D>, dim3(grid), dim3(TA_THREADS),
                                TaSmem<D>::TOTAL, s, 1, qm, km, vm, c, a))
      return rc;
  }
  TraceScope ts("tree.merge", s);
  return launch_k(tree_merge_kernel<D>, dim3(grid, 8), dim3(TM_THREADS), 0, s, 1, c, a, grid);
}

}  // namespace
}  // namespace ivc

using namespace ivc;

extern "C" {

size_t ivc_tree_attention_workspace_size(const ivc_cache* c, int N, int q_heads, int B) {
  if (cache_ok(c) != IVC_OK || N < 0 || B < 0 || B > TA_MAX_BATCH || q_heads < 1) return 0;
  return carve(nullptr, nullptr, B, tree_grid(), c->head_dim);
}

int ivc_tree_attention(const ivc_cache* c, int layer, const void* q, long long q_ld, int N,
                       int q_heads, float scale, const int32_t* parents, const int32_t* offsets,
                       const int32_t* seqs, int B, void* out, void* workspace, size_t ws_bytes,
                       ivc_stream_t stream) {
  if (const int rc = cache_ok(c)) return rc;
  if (layer < 0 || layer >= c->layers || N < 0 || B < 0 || q_heads < 1) return IVC_EINVAL;
  const float scale_log2 = scale * 1.4426950408889634f;  // infinite times a score of 0 is NaN
  if (!(scale > 0.f && scale_log2 < INFINITY)) return IVC_EINVAL;
  if (q_heads % c->kv_heads != 0 || q_heads / c->kv_heads > 64 || B > TA_MAX_BATCH)
    return IVC_EUNSUPPORTED;
  if (q_ld % 8 != 0 || q_ld < static_cast<long long>(q_heads) * c->head_dim) return IVC_EUNSUPPORTED;
  if (!offsets || (N > 0 && (!q || !out))) return IVC_EINVAL;
  auto al = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  if (!al(q) || !al(out)) return IVC_EALIGN;
  if (const int rc = step_ws_ok(workspace, ws_bytes,
                                ivc_tree_attention_workspace_size(c, N, q_heads, B)))
    return rc;
  if (N == 0 || B == 0) return IVC_OK;
  const int D = c->head_dim, grid = tree_grid();
  TreeArgs a = {};
  a.N = N;
  a.q_heads = q_heads;
  a.group = q_heads / c->kv_heads;
  a.npt = TA_ROWS / a.group;
  a.layer = layer;
  a.B = B;
  a.scale_log2 = scale_log2;
  a.parents = parents;
  a.offsets = offsets;
  a.seqs = seqs;
  a.out = static_cast<bf16*>(out);
  a.status = static_cast<int*>(workspace);
  carve(&a, static_cast<char*>(workspace), B, grid, D);
  CUtensorMap qm, km, vm;
  {
    const unsigned long long d[3] = {static_cast<unsigned long long>(D),
                                     static_cast<unsigned long long>(q_heads),
                                     static_cast<unsigned long long>(N)};
    const unsigned long long st[2] = {static_cast<unsigned long long>(D) * 2,
                                      static_cast<unsigned long long>(q_ld) * 2};
    const unsigned box[3] = {64, static_cast<unsigned>(a.group), static_cast<unsigned>(a.npt)};
    if (map_bf16(&qm, 3, q, d, st, box) != IVC_OK) return IVC_ECUDA;
  }
  const size_t rows = static_cast<size_t>(c->pages) * c->kv_heads * c->page_tokens;
  for (int kv = 0; kv < 2; ++kv) {
    const unsigned long long d[2] = {static_cast<unsigned long long>(D), rows};
    const unsigned long long st[1] = {static_cast<unsigned long long>(D) * 2};
    const unsigned box[2] = {64, static_cast<unsigned>(c->page_tokens < TA_KEYS ? c->page_tokens : TA_KEYS)};
    const bf16* base = static_cast<const bf16*>(kv ? c->v : c->k) + rows * D * layer;
    if (map_bf16(kv ? &vm : &km, 2, base, d, st, box) != IVC_OK) return IVC_ECUDA;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return D == 64 ? run_tree<64>(qm, km, vm, *c, a, grid, s) : run_tree<128>(qm, km, vm, *c, a, grid, s);
}

}  // extern "C"
