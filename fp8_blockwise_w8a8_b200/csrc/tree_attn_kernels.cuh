// tree_attn_kernels.cuh -- attention of drafted token trees over the paged FP8 (E4M3) KV cache,
// for sm_100a.
//
// Sequence b has c = ctx_lens[b] committed positions and n = cu[b + 1] - cu[b] drafted nodes,
// cached at positions c .. c + n - 1.  Node i sees the context and the nodes j <= i whose bit j of
// its mask row is set (every j <= i when there is no mask):
//   z_j = sm_scale s_q s_k sum_d dec(q[i][h][d]) dec(k_j[g][d])
//   o[i][h][d] = s_v * sum_j softmax(z)_j dec(v_j[g][d])   -> bf16,   g = h / (Hq / Hkv)
// A node that sees nothing gets zeros.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "attn_kernels.cuh"
#include "ptx.cuh"
#include "spec_kernels.cuh"

namespace fp8q {

struct TreeAttnArgs {
  const uint8_t *q;            // [total][ldq] codes
  int64_t ldq;
  const uint8_t *k_cache, *v_cache;   // [num_slots][Hkv * D]
  int64_t num_blocks;          // num_slots / block_size
  const float *scale3;
  const int32_t *block_table;  // [B][max_blocks]
  int64_t max_blocks;
  const int32_t *ctx_lens, *cu;
  const int64_t *mask;         // [total][ldm] or null
  int64_t ldm;
  int64_t total;
  int B, Hq, Hkv, block_size, max_nodes, max_seq_len;
  float sm_scale;
  uint16_t *out;               // [total][ldo] bf16
  int64_t ldo;
  int row_cap;                 // rows of a partial slot: min(128, max_nodes * Hq / Hkv)
  int32_t *meta;               // [CTAs][kTreeMetaInts]
  float *part;                 // [CTAs][2][row_cap][D + 2]: o, then m, l
};

struct TreeSeq {
  int64_t first;               // row of node 0
  int n, ctx;
};

// The sequence's rows and context, brought into range (recorded where they were not).
__device__ __forceinline__ TreeSeq tree_seq(const TreeAttnArgs &a, int b, bool record) {
  TreeSeq s;
  bool bad;
  s.n = tree_rows(a.cu, b, a.total, a.max_nodes, &s.first, &bad);
  s.ctx = a.ctx_lens[b];
  if (s.ctx < 0 || s.ctx > a.max_seq_len - s.n) {
    bad = true;
    s.ctx = s.ctx < 0 ? 0 : s.ctx;
    s.ctx = s.ctx > a.max_seq_len - s.n ? a.max_seq_len - s.n : s.ctx;
    if (s.ctx < 0) s.ctx = s.n = 0;
  }
  if (bad && record) record_error(9 /* FP8Q_ERR_RANGE */);
  return s;
}

// ---------------------------------------------------------------------------------------------
// Shapes of the kernel
// ---------------------------------------------------------------------------------------------
constexpr int kTreeM = 128;          // query rows (node, head of the group) per row tile: TMEM lanes
constexpr int kTreeN = 64;           // cached positions per tile
constexpr int kTreeThreads = 288;    // 4 softmax warps, 4 load warps, 1 MMA warp
constexpr int kTreeMaxCtas = 296;    // 2 per SM of 148
constexpr int kTreeKStages = 3;      // K tiles in shared memory; 2 in flight ahead of the one in use
constexpr int kTreeAhead = 2;
constexpr int kTreeItemCost = 2;     // cost of starting a row tile, in position tiles
constexpr int kTreeMinCost = 4;      // least cost per CTA
constexpr int kTreeMetaInts = 8;
constexpr float kTreeLag = 8.0f;     // the reference lags the running maximum by at most 2^8
constexpr float kTreeBias = 7.0f;    // weights are 2^(z - reference + 7): at most 2^15 in fp16

template <int D>
struct TreeLayout {
  static constexpr int kQ = 0;                                   // [128][128 B], swizzled
  static constexpr int kK = kQ + kTreeM * 128;                   // [stage][64][128 B], swizzled
  static constexpr int kV16 = kK + kTreeKStages * kTreeN * 128;  // [2][D / 64][64][128 B], swizzled
  static constexpr int kV16Bytes = kTreeN * D * 2;
  static constexpr int kV8 = kV16 + 2 * kV16Bytes;               // [stage][64 * D], by thread
  static constexpr int kSmem = kV8 + kTreeKStages * kTreeN * D + 1024;
  // TMEM columns: scores, two weight buffers (two fp16 a column), values
  static constexpr int kColS = 0, kColP = 64, kColO = 128, kCols = 256;
  static constexpr uint32_t kIdescQK = (1u << 4) | (static_cast<uint32_t>(kTreeN >> 3) << 17) |
                                       (static_cast<uint32_t>(kTreeM >> 4) << 24);
  // kind::f16, fp16 operands, B with its columns (dims) contiguous (bit 16)
  static constexpr uint32_t kIdescPV = (1u << 4) | (1u << 16) |
                                       (static_cast<uint32_t>(D >> 3) << 17) |
                                       (static_cast<uint32_t>(kTreeM >> 4) << 24);
};

// Row tile rt of a sequence with n nodes: its rows, and the position tiles they can see.
__device__ __forceinline__ int tree_row_tiles(int n, int G) {
  return (n * G + kTreeM - 1) / kTreeM;
}
__device__ __forceinline__ int tree_tiles(int n, int ctx, int G, int rt) {
  const int last = (min(n * G, (rt + 1) * kTreeM) - 1) / G;      // the tile's last node
  return (ctx + last) / kTreeN + 1;
}
__device__ __forceinline__ int64_t tree_group_cost(const TreeSeq &s, int G) {
  int64_t c = 0;
  for (int rt = tree_row_tiles(s.n, G) - 1; rt >= 0; --rt)
    c += tree_tiles(s.n, s.ctx, G, rt) + kTreeItemCost;
  return c;
}

// The pieces of work of one CTA: a range of the cost axis on which the items (sequence, kv head, row
// tile) stand one behind the other, each as long as its position tiles plus kTreeItemCost.  A piece
// is the range's share of one item: tiles [t, t_end) of nt.
struct TreeCursor {
  TreeSeq s;
  int64_t rem;
  int B, b, g, rt, t, t_end, nt;
  bool live;

  __device__ __forceinline__ void item(int G, int off) {
    nt = tree_tiles(s.n, s.ctx, G, rt);
    const int cost = nt + kTreeItemCost;
    const int64_t take = min(static_cast<int64_t>(cost - off), rem);
    t = max(0, off - kTreeItemCost);
    t_end = max(0, off + static_cast<int>(take) - kTreeItemCost);
    rem -= take;
  }
  __device__ __forceinline__ void init(const TreeAttnArgs &a, int G, int num, int b0, int64_t off,
                                       int64_t cost) {
    B = num;
    rem = cost;
    live = cost > 0;
    if (!live) return;
    b = b0;
    s = tree_seq(a, b, false);
    const int64_t per_g = tree_group_cost(s, G);
    g = static_cast<int>(off / per_g);
    int64_t o = off - g * per_g;
    for (rt = 0;; ++rt) {
      const int c = tree_tiles(s.n, s.ctx, G, rt) + kTreeItemCost;
      if (o < c) break;
      o -= c;
    }
    item(G, static_cast<int>(o));
    if (t >= t_end) next_piece(a, G);
  }
  __device__ __forceinline__ void next_piece(const TreeAttnArgs &a, int G) {
    do {
      if (rem <= 0) {
        live = false;
        return;
      }
      if (++rt == tree_row_tiles(s.n, G)) {
        rt = 0;
        if (++g == a.Hkv) {
          g = 0;
          do {
            if (++b >= B) {
              live = false;
              return;
            }
            s = tree_seq(a, b, false);
          } while (s.n == 0);
        }
      }
      item(G, 0);
    } while (t >= t_end);
  }
  __device__ __forceinline__ int rows(int G) const { return min(kTreeM, s.n * G - rt * kTreeM); }
};

// Bits of the nodes j0 .. j0 + 63 that node i sees (negative j: the context, seen).
__device__ __forceinline__ uint64_t tree_bits(const int64_t *row, int words, int i, int j0) {
  const int lim = i - j0;                                        // bits above lim lie behind i
  if (lim < 0) return 0ull;
  uint64_t w;
  if (j0 < 0) {
    w = j0 <= -64 ? ~0ull
                  : ((row ? static_cast<uint64_t>(row[0]) : ~0ull) << -j0) | ((1ull << -j0) - 1);
  } else if (row) {
    const int k = j0 >> 6, r = j0 & 63;
    w = k < words ? static_cast<uint64_t>(row[k]) >> r : 0ull;
    if (r && k + 1 < words) w |= static_cast<uint64_t>(row[k + 1]) << (64 - r);
  } else {
    w = ~0ull;
  }
  return lim < 63 ? w & ((2ull << lim) - 1) : w;
}

__device__ __forceinline__ float tree_ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Shared-memory descriptor of fp16 values [position][dim] with 128-byte rows of 64 dims under the
// 128-byte swizzle (dims contiguous): 8-position groups 1024 bytes apart (stride byte offset), the
// next 64 dims 8192 bytes on (leading byte offset).
__device__ __forceinline__ uint64_t tree_sdesc_v(uint32_t saddr) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(8192 >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
         (static_cast<uint64_t>(2) << 61);
}
__device__ __forceinline__ uint64_t tree_sdesc_k(uint32_t saddr) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(1) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
         (static_cast<uint64_t>(2) << 61);
}

template <int N>
__device__ __forceinline__ void tree_ld(uint32_t taddr, uint32_t (&r)[N]) {
  if constexpr (N == 64) tmem_ld_32x32b_x64(taddr, r);
  else if constexpr (N == 32) tmem_ld_32x32b_x32(taddr, r);
  else tmem_ld_32x32b_x16(taddr, r);
  tmem_ld_wait(r);
}
template <int N>
__device__ __forceinline__ void tree_st(uint32_t taddr, const uint32_t (&r)[N]) {
  if constexpr (N == 32) tmem_st_32x32b_x32(taddr, r);
  else if constexpr (N == 16) tmem_st_32x32b_x16(taddr, r);
  else tmem_st_32x32b_x8(taddr, r);
}

// What the CTA's roles share.
struct TreeShared {
  uint64_t k_full[kTreeKStages], v_full[2], s_full, s_free, p_full[2], pv_done[2], sm_sync, drain;
  uint64_t valid[8];             // per tile (mod 8): the positions that exist, one bit each
  int start_b;
  int64_t start_off;
  int64_t warp_sum[kTreeThreads / 32];
  uint32_t tmem;
  int abort;
  int nan_piece;                 // 1 + index of the last piece with a NaN code in V
  float ml[4][32][2];
  float o[4][32][17];
};

// The dims of kv head g that are NaN in a value row seen by row (node i) among the positions of
// [t, t_end) whose column within its tile lies in [c0, c0 + nc).  Runs only where V holds NaN codes.
template <int D>
__device__ __noinline__ uint4 tree_nan_dims(const TreeAttnArgs &a, const TreeCursor &c, int i, int c0,
                                            int nc) {
  uint32_t dims[4] = {};
  const int words = (a.max_nodes + 63) / 64;
  const int64_t *mrow = a.mask ? a.mask + (c.s.first + i) * a.ldm : nullptr;
  for (int tile = c.t; tile < c.t_end; ++tile) {
    const uint64_t bits = tree_bits(mrow, words, i, tile * kTreeN - c.s.ctx);
    for (int col = c0; col < c0 + nc; ++col) {
      const int pos = tile * kTreeN + col;
      if (!((bits >> col) & 1) || pos >= c.s.ctx + c.s.n) continue;
      const int32_t blk = a.block_table[c.b * a.max_blocks + pos / a.block_size];
      if (blk < 0 || blk >= a.num_blocks) continue;
      const int64_t slot = static_cast<int64_t>(blk) * a.block_size + pos % a.block_size;
      const uint32_t *v = reinterpret_cast<const uint32_t *>(a.v_cache + (slot * a.Hkv + c.g) * D);
#pragma unroll
      for (int w = 0; w < D / 32; ++w)
        for (int x = 0; x < 8; ++x) {
          const uint32_t word = v[8 * w + x];
          for (int y = 0; y < 4; ++y)
            if (((word >> (8 * y)) & 0x7F) == 0x7F) dims[w] |= 1u << (4 * x + y);
        }
    }
  }
  return make_uint4(dims[0], dims[1], dims[2], dims[3]);
}

// One row tile's running state in a softmax thread.
struct TreeRow {
  float ref, l;                  // reference of the weights (log2 units), their sum
};

// One position tile: the scores of NC columns of this thread's row become weights in TMEM.
template <int D, int NC>
__device__ __forceinline__ bool tree_tile(TreeShared &sh, uint32_t tmem, uint32_t col0, uint32_t it,
                                          bool first, uint64_t seen, float c2, TreeRow &st) {
  using L = TreeLayout<D>;
  const int lane = threadIdx.x & 31;
  if (!wait_warp(smem_u32(&sh.s_full), it & 1u, &sh.abort)) return false;
  tc_fence_after();
  uint32_t sr[NC];
  tree_ld<NC>(tmem + L::kColS + col0, sr);
  seen &= sh.valid[it & 7u];
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(smem_u32(&sh.s_free));
  const uint64_t mine = seen >> col0;
  const uint64_t all = NC == 64 ? ~0ull : (1ull << (NC & 63)) - 1;
  if (!__all_sync(0xffffffffu, (mine & all) == all)) {
#pragma unroll
    for (int j = 0; j < NC; ++j)
      if (!((mine >> j) & 1)) sr[j] = 0xFF800000u;               // -inf
  }
  float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int j = 0; j < NC; ++j) mx[j & 3] = fmaxf(mx[j & 3], __uint_as_float(sr[j]));
  const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c2;
  // P buffer it & 1 was read by the MMA of tile it - 2
  if (it >= 2 && !wait_warp(smem_u32(&sh.pv_done[it & 1u]), ((it - 2) >> 1) & 1u, &sh.abort))
    return false;
  const bool up = top > st.ref + kTreeLag;                       // also the first score seen
  if (__any_sync(0xffffffffu, up)) {
    const bool held = up && st.ref != -INFINITY;                 // values to rescale
    const float f = up ? tree_ex2(st.ref - top) : 1.0f;          // 0 from -inf
    st.ref = up ? top : st.ref;
    st.l *= f;
    if (!first && __any_sync(0xffffffffu, held)) {
      if (!wait_warp(smem_u32(&sh.pv_done[(it - 1) & 1u]), ((it - 1) >> 1) & 1u, &sh.abort))
        return false;
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < D; c += 16) {
        uint32_t o[16];
        tree_ld<16>(tmem + L::kColO + c, o);
#pragma unroll
        for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
        tree_st<16>(tmem + L::kColO + c, o);
      }
    }
  }
  const float bias = kTreeBias - (st.ref == -INFINITY ? 0.0f : st.ref);
  float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  uint32_t pk[NC / 2];
#pragma unroll
  for (int j = 0; j < NC; j += 2) {
    const float p0 = tree_ex2(fmaf(__uint_as_float(sr[j]), c2, bias));
    const float p1 = tree_ex2(fmaf(__uint_as_float(sr[j + 1]), c2, bias));
    sum[j & 3] += p0;
    sum[(j & 3) + 1] += p1;
    pk[j / 2] = f32x2_to_f16x2(p0, p1);
  }
  st.l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
  tree_st<NC / 2>(tmem + L::kColP + 32 * (it & 1u) + col0 / 2, pk);
  tmem_st_wait();
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(smem_u32(&sh.p_full[it & 1u]));
  return true;
}

// Bounded barrier of the four softmax warps.
__device__ __forceinline__ bool tree_sync4(TreeShared &sh, uint32_t &phase) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&sh.sm_sync));
  const bool ok = wait_warp(smem_u32(&sh.sm_sync), phase & 1u, &sh.abort);
  ++phase;
  return ok;
}

template <int D>
__global__ void __launch_bounds__(kTreeThreads, 2) k_tree_attn(const TreeAttnArgs a) {
  using L = TreeLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ TreeShared sh;
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.Hq / a.Hkv;

  if (tid == 0) {
    for (int i = 0; i < kTreeKStages; ++i) mbar_init(smem_u32(&sh.k_full[i]), 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sh.v_full[i]), 4);
      mbar_init(smem_u32(&sh.p_full[i]), 4);
      mbar_init(smem_u32(&sh.pv_done[i]), 1);
    }
    mbar_init(smem_u32(&sh.s_full), 1);
    mbar_init(smem_u32(&sh.s_free), 4);
    mbar_init(smem_u32(&sh.sm_sync), 4);
    mbar_init(smem_u32(&sh.drain), 1);
    sh.abort = 0;
    sh.nan_piece = 0;
    fence_barrier_init();
  }
  if (warp == 8) {
    tmem_alloc(smem_u32(&sh.tmem), L::kCols);
    tmem_relinquish();
  }

  // This CTA's range of the cost axis: every CTA adds up all sequences' costs itself.  Offsets that
  // decrease end the batch before that sequence, so that no two sequences write the same rows.
  const int per = (a.B + kTreeThreads - 1) / kTreeThreads;
  int B = a.B;
  int64_t mine, upto, total;
  for (bool again = false;; again = true) {
    mine = 0;
    bool falls = false;
    for (int b = tid * per; b < min(B, (tid + 1) * per); ++b) {
      falls |= a.cu[b + 1] < a.cu[b];
      mine += tree_group_cost(tree_seq(a, b, blockIdx.x == 0), G) * a.Hkv;
    }
    upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += y;
    }
    if (lane == 31) sh.warp_sum[warp] = upto;
    if (!__syncthreads_or(falls) || again) break;
    if (tid == 0) sh.start_b = a.B;
    __syncthreads();
    for (int b = tid * per; b < min(B, (tid + 1) * per); ++b)
      if (a.cu[b + 1] < a.cu[b]) {
        atomicMin(&sh.start_b, b);
        break;
      }
    __syncthreads();
    B = sh.start_b;
    __syncthreads();
  }
  total = 0;
  for (int w = 0; w < kTreeThreads / 32; ++w) {
    if (w < warp) upto += sh.warp_sum[w];
    total += sh.warp_sum[w];
  }
  const int64_t most = (total + kTreeMinCost - 1) / kTreeMinCost;
  const int64_t ctas = most < gridDim.x ? most : gridDim.x;
  const bool works = blockIdx.x < ctas;
  const int64_t lo = works ? total * blockIdx.x / ctas : 0;
  const int64_t hi = works ? total * (blockIdx.x + 1) / ctas : 0;
  int32_t *meta = a.meta + blockIdx.x * kTreeMetaInts;
  if (tid == 0) meta[0] = meta[1] = 0;
  if (works && lo >= upto - mine && lo < upto) {
    int64_t off = lo - (upto - mine);
    int b = tid * per;
    for (;; ++b) {
      const int64_t c = tree_group_cost(tree_seq(a, b, false), G) * a.Hkv;
      if (off < c) break;
      off -= c;
    }
    sh.start_b = b;
    sh.start_off = off;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;

  if (warp >= 4 && warp < 8) {
    // ---------------------------------------------------------------- load and convert
    constexpr int NR = D / 32;                                   // rows of a tile per thread
    constexpr int LPR = D / 16;                                  // lanes per row
    const int lw = warp - 4, lt = tid - 128, ch = lane % LPR;
    const int64_t row = static_cast<int64_t>(a.Hkv) * D;
    const float c = a.sm_scale * a.scale3[0] * a.scale3[1];
    const uint32_t qflip = c < 0.0f ? 0x80808080u : 0u;          // a negative scale negates Q
    TreeCursor pre, cur;
    if (works) pre.init(a, G, B, sh.start_b, sh.start_off, hi - lo);
    pre.live = works && pre.live;
    cur = pre;
    int32_t blk[NR];
    int off[NR];
    // block ids of the prefetch cursor's tile
    auto look_up = [&]() {
      if (!pre.live) return;
#pragma unroll
      for (int j = 0; j < NR; ++j) {
        const int pos = pre.t * kTreeN + 16 * lw + j * (32 / LPR) + lane / LPR;
        const int q = pos / a.block_size;
        off[j] = pos - q * a.block_size;
        blk[j] = -1;
        if (pos < pre.s.ctx + pre.s.n) blk[j] = a.block_table[pre.b * a.max_blocks + q];
        else off[j] = -1;                                        // behind the sequence
      }
    };
    uint32_t pit = 0;                                            // tiles issued
    auto issue = [&]() {
      if (pre.live) {
        const uint32_t st = pit % kTreeKStages;
        uint32_t bits = 0;
#pragma unroll
        for (int j = 0; j < NR; ++j) {
          const int p = 16 * lw + j * (32 / LPR) + lane / LPR;
          const bool there = blk[j] >= 0 && blk[j] < a.num_blocks;
          if (!there && off[j] >= 0) record_error(9 /* FP8Q_ERR_RANGE */);
          const int64_t at =
              there ? (static_cast<int64_t>(blk[j]) * a.block_size + off[j]) * row + pre.g * D + ch * 16
                    : 0;
          const uint32_t nb = there ? 16u : 0u;
          cp_async16(sbase + L::kK + st * kTreeN * 128 + p * 128 + ((ch ^ (p & 7)) << 4),
                     a.k_cache + at, nb);
          cp_async16(sbase + L::kV8 + st * kTreeN * D + (j * 128 + lt) * 16, a.v_cache + at, nb);
          bits |= there ? 1u << (p & 15) : 0u;
        }
        bits = __reduce_or_sync(0xffffffffu, bits);
        if (lane == 0)
          reinterpret_cast<uint16_t *>(&sh.valid[pit & 7u])[lw] = static_cast<uint16_t>(bits);
        ++pit;
        if (++pre.t >= pre.t_end) pre.next_piece(a, G);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      look_up();
    };
    look_up();
#pragma unroll
    for (int i = 0; i < kTreeAhead; ++i) issue();
    bool fresh = true, ok = true;
    int piece = 0;
    for (uint32_t it = 0; cur.live; ++it) {
      const uint32_t st = it % kTreeKStages;
      if (fresh) {
        // Q rows of the piece, once the scores of the piece before are complete: row r is head
        // g G + r % G of node r / G; up to 32 (64) rows are repeated 4 (2) times down the tile
        if (it > 0 && !wait_warp(smem_u32(&sh.s_full), (it - 1) & 1u, &sh.abort)) { ok = false; break; }
        const int rows = cur.rows(G), step = rows <= 32 ? 32 : (rows <= 64 ? 64 : 128);
        for (int i = lt; i < kTreeM * LPR; i += 128) {
          const int r = i / LPR, c16 = i % LPR, rr = r % step;
          uint4 v = make_uint4(0, 0, 0, 0);
          if (rr < rows) {
            const int idx = cur.rt * kTreeM + rr, node = idx / G, h = cur.g * G + idx % G;
            v = *reinterpret_cast<const uint4 *>(a.q + (cur.s.first + node) * a.ldq + h * D + c16 * 16);
            v.x ^= qflip; v.y ^= qflip; v.z ^= qflip; v.w ^= qflip;
          }
          *reinterpret_cast<uint4 *>(smem + L::kQ + r * 128 + ((c16 ^ (r & 7)) << 4)) = v;
        }
        fresh = false;
        ++piece;
      }
      asm volatile("cp.async.wait_group %0;" ::"n"(kTreeAhead - 1) : "memory");
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.k_full[st]));
      // the K stage of tile it - 1 is free once its scores are complete
      if (it > 0 && !wait_warp(smem_u32(&sh.s_full), (it - 1) & 1u, &sh.abort)) { ok = false; break; }
      uint4 v8[NR];
#pragma unroll
      for (int j = 0; j < NR; ++j)
        v8[j] = *reinterpret_cast<const uint4 *>(smem + L::kV8 + st * kTreeN * D + (j * 128 + lt) * 16);
      issue();
      if (it >= 2 && !wait_warp(smem_u32(&sh.pv_done[it & 1u]), ((it - 2) >> 1) & 1u, &sh.abort)) {
        ok = false;
        break;
      }
      // V codes to fp16 (exact); a NaN code becomes 0 here and is put back where it is seen
      uint8_t *v16 = smem + L::kV16 + (it & 1u) * L::kV16Bytes;
      bool nan = false;
#pragma unroll
      for (int j = 0; j < NR; ++j) {
        const int p = 16 * lw + j * (32 / LPR) + lane / LPR;
        uint32_t w[4] = {v8[j].x, v8[j].y, v8[j].z, v8[j].w};
        uint32_t h[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t n7 = ((w[k] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
          if (n7) {
            nan = true;
            w[k] &= ~((n7 >> 7) * 0xFFu);
          }
          h[2 * k] = e4m3x2_to_f16x2(w[k] & 0xFFFFu);
          h[2 * k + 1] = e4m3x2_to_f16x2(w[k] >> 16);
        }
        // the halves of a row's dims are stored in opposite order, so that a quarter warp covers
        // all banks
        const int half = D == 128 ? ch >> 2 : 0, c0 = (ch & 3) * 2;
        uint8_t *dst = v16 + half * 8192 + p * 128;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int e = k ^ half;
          *reinterpret_cast<uint4 *>(dst + (((c0 + e) ^ (p & 7)) << 4)) =
              e ? make_uint4(h[4], h[5], h[6], h[7]) : make_uint4(h[0], h[1], h[2], h[3]);
        }
      }
      if (nan) atomicMax(&sh.nan_piece, piece);
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.v_full[it & 1u]));
      if (++cur.t >= cur.t_end) {
        cur.next_piece(a, G);
        fresh = true;
      }
    }
    (void)ok;
    asm volatile("cp.async.wait_group 0;" ::: "memory");         // none in flight at exit
  } else if (warp == 8) {
    // ---------------------------------------------------------------- MMA issue
    if (lane == 0) {
      TreeCursor cur;
      if (works) cur.init(a, G, B, sh.start_b, sh.start_off, hi - lo);
      cur.live = works && cur.live;
      const uint64_t qd = tree_sdesc_k(sbase + L::kQ);
      auto scores = [&](uint32_t it) {
        const uint32_t st = it % kTreeKStages;
        if (!wait_one(smem_u32(&sh.k_full[st]), (it / kTreeKStages) & 1u, &sh.abort)) return false;
        tc_fence_after();
        const uint64_t kd = tree_sdesc_k(sbase + L::kK + st * kTreeN * 128);
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk)
          mma_f8f6f4(tmem + L::kColS, qd + 2 * kk, kd + 2 * kk, L::kIdescQK, kk > 0 ? 1u : 0u);
        mma_commit(smem_u32(&sh.s_full));
        return true;
      };
      bool ok = !cur.live || scores(0), first = true;
      for (uint32_t it = 0; cur.live && ok; ++it) {
        const bool fresh = first;
        first = false;
        if (++cur.t >= cur.t_end) {
          cur.next_piece(a, G);
          first = true;
        }
        if (cur.live)
          ok = wait_one(smem_u32(&sh.s_free), it & 1u, &sh.abort) && scores(it + 1);
        if (!ok || !wait_one(smem_u32(&sh.p_full[it & 1u]), (it >> 1) & 1u, &sh.abort) ||
            !wait_one(smem_u32(&sh.v_full[it & 1u]), (it >> 1) & 1u, &sh.abort))
          break;
        tc_fence_after();
        const uint64_t vd = tree_sdesc_v(sbase + L::kV16 + (it & 1u) * L::kV16Bytes);
#pragma unroll
        for (int kk = 0; kk < kTreeN / 16; ++kk)
          mma_f16_ts(tmem + L::kColO, tmem + L::kColP + 32 * (it & 1u) + 8 * kk, vd + 128 * kk,
                     L::kIdescPV, fresh && kk == 0 ? 0u : 1u);
        mma_commit(smem_u32(&sh.pv_done[it & 1u]));
      }
      mma_commit(smem_u32(&sh.drain));                           // all MMAs done before dealloc
      wait_drain(smem_u32(&sh.drain), 0);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- softmax and output
    TreeCursor cur;
    if (works) cur.init(a, G, B, sh.start_b, sh.start_off, hi - lo);
    cur.live = works && cur.live;
    float c2 = fabsf(a.sm_scale * a.scale3[0] * a.scale3[1]) * 1.4426950408889634f;
    c2 = c2 < 1e-37f ? 1e-37f : c2;                              // so that -inf stays -inf
    const float sv = a.scale3[2];
    const uint32_t tw = tmem + (static_cast<uint32_t>(32 * warp) << 16);
    const int words = (a.max_nodes + 63) / 64;
    uint32_t it = 0, phase = 0;
    int piece = 0;
    bool ok = true;
    for (; cur.live && ok; cur.next_piece(a, G)) {
      ++piece;
      const int rows = cur.rows(G), rep = rows <= 32 ? 4 : (rows <= 64 ? 2 : 1);
      const int r = rep == 4 ? lane : (rep == 2 ? 32 * (warp & 1) + lane : 32 * warp + lane);
      const int nc = kTreeN / rep;
      const uint32_t col0 = rep == 4 ? 16 * warp : (rep == 2 ? 32 * (warp >> 1) : 0);
      const bool live = r < rows;
      const int node = (cur.rt * kTreeM + r) / G;
      const int64_t *mrow = a.mask && live ? a.mask + (cur.s.first + node) * a.ldm : nullptr;
      if (rep > 1) {                                             // weights of the other columns: 0
        const uint32_t z[32] = {};
        tree_st<32>(tw + L::kColP, z);
        tree_st<32>(tw + L::kColP + 32, z);
      }
      TreeRow st{-INFINITY, 0.0f};
      for (int t = cur.t; t < cur.t_end && ok; ++t, ++it) {
        // a row that does not exist counts as seeing all (its scores are 0, its results unused)
        const uint64_t seen = live ? tree_bits(mrow, words, node, t * kTreeN - cur.s.ctx) : ~0ull;
        const bool first = t == cur.t;
        ok = rep == 4   ? tree_tile<D, 16>(sh, tw, col0, it, first, seen, c2, st)
             : rep == 2 ? tree_tile<D, 32>(sh, tw, col0, it, first, seen, c2, st)
                        : tree_tile<D, 64>(sh, tw, col0, it, first, seen, c2, st);
      }
      if (!ok || !wait_warp(smem_u32(&sh.pv_done[(it - 1) & 1u]), ((it - 1) >> 1) & 1u, &sh.abort))
        break;
      tc_fence_after();
      uint4 nan = make_uint4(0, 0, 0, 0);
      const bool any_nan = *reinterpret_cast<volatile int *>(&sh.nan_piece) >= piece;
      if (any_nan && live) nan = tree_nan_dims<D>(a, cur, node, col0, nc);
      auto is_nan = [&](int d) {
        const uint32_t w = d < 64 ? (d < 32 ? nan.x : nan.y) : (d < 96 ? nan.z : nan.w);
        return ((w >> (d & 31)) & 1) != 0;
      };
      const bool whole = cur.t == 0 && cur.t_end == cur.nt;
      const int slot = cur.t > 0 ? 0 : 1;
      float *part = a.part + (static_cast<int64_t>(blockIdx.x) * 2 + slot) * a.row_cap * (D + 2);
      float *ml = part + static_cast<int64_t>(a.row_cap) * D;
      if (warp == 0 && lane == 0 && !whole) {
        if (slot == 0) meta[0] = cur.t_end == cur.nt ? 2 : 1;    // a part; 2: the item's last
        else {
          meta[1] = 1;                                           // the item's first part
          meta[2] = static_cast<int>(cur.s.first);
          meta[3] = cur.rt * kTreeM;
          meta[4] = rows;
          meta[5] = cur.g;
        }
      }
      if (rep == 1) {
        const float f = whole ? (st.l == 0.0f ? 0.0f : sv / st.l) : 1.0f;
        const int h = cur.g * G + (cur.rt * kTreeM + r) % G;
        uint16_t *out = a.out + (cur.s.first + node) * a.ldo + h * D;
#pragma unroll
        for (int c = 0; c < D; c += 16) {
          uint32_t o[16];
          tree_ld<16>(tw + L::kColO + c, o);
          float v[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            v[j] = st.l == 0.0f ? 0.0f : __uint_as_float(o[j]) * f;
            if (is_nan(c + j)) v[j] = NAN;
          }
          if (!live) continue;
          if (whole) {
            uint32_t pk[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const __nv_bfloat162 b2 = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
              pk[j] = *reinterpret_cast<const uint32_t *>(&b2);
            }
            *reinterpret_cast<uint4 *>(out + c) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
            *reinterpret_cast<uint4 *>(out + c + 8) = make_uint4(pk[4], pk[5], pk[6], pk[7]);
          } else {
#pragma unroll
            for (int j = 0; j < 16; j += 4)
              *reinterpret_cast<float4 *>(part + r * D + c + j) =
                  make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
          }
        }
        if (live && !whole) {
          ml[2 * r] = st.ref;
          ml[2 * r + 1] = st.l;
        }
      } else {
        // the repeats of a row hold different positions: merge them
        sh.ml[warp][lane][0] = st.ref;
        sh.ml[warp][lane][1] = st.l;
        if (!tree_sync4(sh, phase)) break;
        auto merged = [&](int w0, int ln, float &M, float &l) {
          M = -INFINITY;
          l = 0.0f;
          for (int w = w0; w < 4; w += 4 / rep) M = fmaxf(M, sh.ml[w][ln][0]);
          for (int w = w0; w < 4; w += 4 / rep) {
            const float m = sh.ml[w][ln][0];
            l += sh.ml[w][ln][1] * (m == M ? 1.0f : tree_ex2(m - M));
          }
        };
        float M, l;
        merged(rep == 4 ? 0 : warp & 1, lane, M, l);
        const float f = st.ref == M ? 1.0f : tree_ex2(st.ref - M);
        // summed by rows: `rep` threads per row, 16 / rep columns each
        const int tr = tid / rep, tc = (tid % rep) * (16 / rep);
        float tM, tl;
        merged(rep == 4 ? 0 : tr / 32, tr % 32, tM, tl);
        const float scale = whole ? (tl == 0.0f ? 0.0f : sv / tl) : 1.0f;
        const int idx = cur.rt * kTreeM + tr, h = cur.g * G + idx % G;
        uint16_t *out = a.out + (cur.s.first + idx / G) * a.ldo + h * D + tc;
        for (int c = 0; c < D && ok; c += 16) {
          uint32_t o[16];
          tree_ld<16>(tw + L::kColO + c, o);
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float v = st.l == 0.0f ? 0.0f : __uint_as_float(o[j]) * f;
            if (is_nan(c + j)) v = NAN;
            sh.o[warp][lane][j] = v;
          }
          if (!tree_sync4(sh, phase)) { ok = false; break; }
          if (tr < rows) {
            for (int j = 0; j < 16 / rep; j += 4) {
              float v[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                float x = 0.0f;
                for (int w = rep == 4 ? 0 : tr / 32; w < 4; w += 4 / rep)
                  x += sh.o[w][tr % 32][tc + j + k];
                v[k] = x * scale;
              }
              if (whole) {
                const __nv_bfloat162 b0 = __floats2bfloat162_rn(v[0], v[1]);
                const __nv_bfloat162 b1 = __floats2bfloat162_rn(v[2], v[3]);
                *reinterpret_cast<uint2 *>(out + c + j) =
                    make_uint2(*reinterpret_cast<const uint32_t *>(&b0),
                               *reinterpret_cast<const uint32_t *>(&b1));
              } else {
                *reinterpret_cast<float4 *>(part + tr * D + c + tc + j) =
                    make_float4(v[0], v[1], v[2], v[3]);
              }
            }
          }
          if (!tree_sync4(sh, phase)) { ok = false; break; }
        }
        if (!whole && tr < rows && tc == 0) {
          ml[2 * tr] = tM;
          ml[2 * tr + 1] = tl;
        }
      }
      tc_fence_before();
    }
  }

  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kCols);
  }
}

// The items that several CTAs shared: block (i, y) takes the rows 8 y .. 8 y + 7 of the item whose
// first part is CTA i's last piece, and adds the parts in CTA order, each a running maximum's state.
template <int D>
__global__ void __launch_bounds__(256) k_tree_attn_combine(const TreeAttnArgs a) {
  constexpr int V = D / 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int i = blockIdx.x;
  const int32_t *meta = a.meta + i * kTreeMetaInts;
  if (meta[1] == 0) return;
  const int r = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (r >= meta[4]) return;
  const int G = a.Hq / a.Hkv, idx = meta[3] + r, h = meta[5] * G + idx % G;
  const int64_t slot = static_cast<int64_t>(a.row_cap) * (D + 2);
  float M = -INFINITY, l = 0.0f, o[V] = {};
  for (int j = i;; ++j) {
    const float *part = a.part + (2 * static_cast<int64_t>(j) + (j == i ? 1 : 0)) * slot;
    const float m = part[static_cast<int64_t>(a.row_cap) * D + 2 * r];
    const float lj = part[static_cast<int64_t>(a.row_cap) * D + 2 * r + 1];
    if (lj != 0.0f) {
      const float top = fmaxf(M, m);
      const float f = M == top ? 1.0f : tree_ex2(M - top), fj = m == top ? 1.0f : tree_ex2(m - top);
      l = l * f + lj * fj;
#pragma unroll
      for (int v = 0; v < V; ++v) o[v] = o[v] * f + part[r * D + V * lane + v] * fj;
      M = top;
    }
    if (j > i && a.meta[j * kTreeMetaInts] != 1) break;
    if (j + 1 >= static_cast<int>(gridDim.x)) break;
  }
  const float f = l == 0.0f ? 0.0f : a.scale3[2] / l;
  uint16_t *out = a.out + (static_cast<int64_t>(meta[2]) + idx / G) * a.ldo + h * D + V * lane;
#pragma unroll
  for (int v = 0; v < V; v += 2) {
    const __nv_bfloat162 b2 = __floats2bfloat162_rn(l == 0.0f ? 0.0f : o[v] * f,
                                                    l == 0.0f ? 0.0f : o[v + 1] * f);
    *reinterpret_cast<uint32_t *>(out + v) = *reinterpret_cast<const uint32_t *>(&b2);
  }
}

}  // namespace fp8q
