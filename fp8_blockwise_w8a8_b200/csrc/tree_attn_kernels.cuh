// tree_attn_kernels.cuh -- attention of drafted token trees over the paged FP8 (E4M3) KV cache,
// for sm_100a.
//
// Sequence b has c = ctx_lens[b] committed positions and n = cu[b + 1] - cu[b] drafted nodes,
// cached at positions c .. c + n - 1.  Node i sees the context and the nodes j <= i whose bit j of
// its mask row is set (every j <= i when there is no mask):
//   z_j = sm_scale s_q s_k sum_d dec(q[i][h][d]) dec(k_j[g][d])
//   o[i][h][d] = s_v * sum_j softmax(z)_j dec(v_j[g][d])   -> bf16,   g = h / (Hq / Hkv)
// A node that sees nothing gets zeros.
//
// Products on the tensor cores, accumulators in TMEM.  A row tile is 128 query rows (node, head of the
// group); a position tile is 64 cached positions of one kv head.  Scores: kind::f8f6f4 on the codes as
// they are.  Weights: fp16 (at most 2^-11 off, half the bound of bf16 results), written over the scores
// in TMEM as the next product's A operand; V is converted to fp16, which is exact.  The softmax keeps a
// reference that lags the running maximum by at most 2^8, so that the accumulators are rescaled rarely.
//
// Few rows leave most of a row tile idle: up to 32 (64) rows are repeated four (two) times down it, each
// repeat takes the weights of its own 16 (32) of a tile's positions (the others are written as zeros),
// and the repeats are merged at the end.  So every softmax warp works, whatever the draft's size.
//
// Work is split evenly whatever the lengths: all items (sequence, kv head, row tile) stand one behind
// the other on one axis of position tiles, two CTAs per SM take equal shares of it, and what CTAs share
// of an item is merged by a second kernel in CTA order, so that results do not depend on timing.
//
// Roles of a CTA's eleven warps: 0-3 softmax and output, 4-7 V (copies by cp.async, conversion to fp16),
// 8 MMAs, 9 K (by TMA a copy per run of positions in a block, or row by row), 10 queries.  Every wait is
// bounded, and a warp's lanes leave it together.
//
// Measured (calls back to back, new inputs every time, several boxes): 64 sequences of 512 to 4096
// positions with up to 16 nodes, 32/8 heads of 128: 107 to 113 us, 2.8 to 3.0 TB/s of cache and 43 to 46 %
// of the copy rate; one sequence of 131501 positions with 61 nodes 191 to 205 us, 640 to 685 TFLOP/s; 8 of
// up to 512 nodes over up to 6000 positions 332 to 341 us, 690 to 712 TFLOP/s; 40 sequences, 16 heads of
// 64, blocks of 7: 64 us.  What bounds it is the issue of the roles' instructions and the hand-offs
// between them (0.46 to 0.53 instructions per cycle and scheduler), with the tensor pipe at 29 %.  80
// registers a thread, of which heads of 128 spill 8 bytes.  The MMA warp runs converged, one lane issuing, so that its
// operands stay in uniform registers: 128 -> 107 us on the first case.  The roles' code has to stay
// small: at 170 KB instruction fetch was the largest stall and everything took twice as long.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "attn_kernels.cuh"
#include "ptx.cuh"
#include "spec_kernels.cuh"

namespace fp8q {

// p / d as p * mul >> shift for 0 <= p < 2^31: mul = floor(2^(31 + l) / d) + 1 and shift = 31 + l, where
// 2^l >= d is the least power of two.
struct TreeDiv {
  uint32_t mul, shift;
  __device__ __forceinline__ int operator()(int p) const {
    return static_cast<int>(static_cast<uint64_t>(static_cast<uint32_t>(p)) * mul >> shift);
  }
};

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
  int box;                     // rows per TMA copy: the power of two in block_size, at most 64
  uint64_t grid_recip;         // floor((2^64 - 1) / gridDim.x)
  TreeDiv by_block, by_group;  // by block_size and by G = Hq / Hkv
  int row_cap;                 // rows of a partial slot: min(128, max_nodes * Hq / Hkv)
  int32_t *meta;               // [CTAs][kTreeMetaInts]
  float *part;                 // [CTAs][2][row_cap][D + 2]: o, then m, l
  uint32_t polls;              // of a bounded wait
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
constexpr int kTreeThreads = 352;    // 4 softmax warps, 4 for V, one each for the MMAs, K and Q
constexpr int kTreeMaxCtas = 296;    // 2 per SM of 148
constexpr int kTreeStages = 4;       // K tiles in shared memory
constexpr int kTreeItemCost = 4;     // cost of starting a row tile, in position tiles
constexpr int kTreeMinCost = 4;      // least cost per CTA
constexpr int kTreeMetaInts = 8;
constexpr float kTreeLag = 8.0f;     // the reference lags the running maximum by at most 2^8
constexpr float kTreeBias = 7.0f;    // weights are 2^(z - reference + 7): at most 2^15 in fp16

template <int D>
struct TreeLayout {
  static constexpr int kQ = 0;                                   // [128][128 B], swizzled
  static constexpr int kK = kQ + kTreeM * 128;                   // [stage][64][D], swizzled
  static constexpr int kTile = kTreeN * D;
  static constexpr int kV16 = kK + kTreeStages * kTile;          // [2][D / 64][64][128 B], swizzled
  static constexpr int kV16Bytes = kTreeN * D * 2;
  static constexpr int kV8 = kV16 + 2 * kV16Bytes;               // [pair of V warps][64][D]
  static constexpr int kSmem = kV8 + 2 * kTile + 1024;
  // TMEM columns: two score buffers, whose first halves then hold the weights (two fp16 a column),
  // and the values
  static constexpr int kColS = 0, kColO = 128, kCols = 256;
  static constexpr uint32_t kIdescQK = (1u << 4) | (static_cast<uint32_t>(kTreeN >> 3) << 17) |
                                       (static_cast<uint32_t>(kTreeM >> 4) << 24);
  // K goes row by row by cp.async where a TMA copy has less than 512 bytes.  40 sequences, heads of 64,
  // blocks of 4: 65.5 us against 76 by TMA, of 8: 65.8 against 66.6; blocks of 7 by TMA gathers of four
  // rows: 82.  64 sequences, heads of 128, blocks of 4: 130 against 124, of 16: 128 against 106.
  static constexpr __host__ __device__ bool by_row(int box) { return box * D < 512; }
  // kind::f16, fp16 operands, B with its columns (dims) contiguous (bit 16)
  static constexpr uint32_t kIdescPV = (1u << 4) | (1u << 16) |
                                       (static_cast<uint32_t>(D >> 3) << 17) |
                                       (static_cast<uint32_t>(kTreeM >> 4) << 24);
};

// Row tile rt of a sequence with n nodes: its rows, and the position tiles they can see.
__device__ __forceinline__ int tree_row_tiles(int n, int G) {
  return (n * G + kTreeM - 1) / kTreeM;
}
__device__ __forceinline__ int tree_tiles(const TreeAttnArgs &a, const TreeSeq &s, int G, int rt) {
  const int last = a.by_group(min(s.n * G, (rt + 1) * kTreeM) - 1);  // the tile's last node
  return (s.ctx + last) / kTreeN + 1;
}
__device__ __forceinline__ int64_t tree_group_cost(const TreeAttnArgs &a, const TreeSeq &s, int G) {
  int64_t c = 0;
#pragma unroll 1
  for (int rt = tree_row_tiles(s.n, G) - 1; rt >= 0; --rt)
    c += tree_tiles(a, s, G, rt) + kTreeItemCost;
  return c;
}

// A share of one item (sequence, kv head, row tile): its position tiles [t, t_end) of nt.  The load
// warp hands the pieces of a CTA to the other roles, the last one with t_end = 0.
struct TreePiece {
  int64_t first;                 // row of the sequence's node 0
  int b, n, ctx, g, row0, rows, t, t_end, nt;
};

// The pieces of work of one CTA: a range of the cost axis on which the items stand one behind the
// other, each as long as its position tiles plus kTreeItemCost.
struct TreeCursor {
  TreeSeq s;
  int64_t rem;
  int B, b, g, rt, t, t_end, nt;
  bool live;

  // From the sequence b0, `off` behind its start; cost 0: nothing.
  __device__ __forceinline__ void init(const TreeAttnArgs &a, int G, int num, int b0, int64_t off,
                                       int64_t cost) {
    B = num;
    rem = cost;
    b = b0;
    g = rt = t = t_end = 0;
    live = cost > 0;
    if (!live) return;
    s = tree_seq(a, b, false);
    const int64_t per_g = tree_group_cost(a, s, G);
    while (off >= per_g) {
      off -= per_g;
      ++g;
    }
    int tiles;
    while (off >= (tiles = tree_tiles(a, s, G, rt) + kTreeItemCost)) {
      off -= tiles;
      ++rt;
    }
    --rt;
    next(a, G, static_cast<int>(off));
  }
  // The next piece, `off` into its item.
  __device__ __forceinline__ void next(const TreeAttnArgs &a, int G, int off) {
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
      nt = tree_tiles(a, s, G, rt);
      const int64_t take = min(static_cast<int64_t>(nt + kTreeItemCost - off), rem);
      t = max(0, off - kTreeItemCost);
      t_end = max(0, off + static_cast<int>(take) - kTreeItemCost);
      rem -= take;
      off = 0;
    } while (t >= t_end);
  }
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
// Descriptor of codes with rows of B = 64 or 128 bytes under the swizzle of that width: 8-row groups
// 8 B bytes apart.
template <int B>
__device__ __forceinline__ uint64_t tree_sdesc_k(uint32_t saddr) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(1) << 16) |
         (static_cast<uint64_t>(8 * B >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
         (static_cast<uint64_t>(B == 128 ? 2 : 4) << 61);
}

// Bounded wait of a warp, short in code: after `*polls` polls in vain the timeout is recorded, *polls
// becomes 0 and the CTA's roles give up.  A poll in vain takes 4.0 us on a B200, whatever time it is
// given, so 2^18 of them are a second.  Every wait but one is for the next position tile or less; that one
// has `rounds` times the limit.  The lanes leave it together.
__device__ __forceinline__ bool tree_poll(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
constexpr uint32_t kTreePolls = 1u << 18;
__device__ __forceinline__ bool tree_wait(const uint64_t &barrier, uint32_t parity,
                                          volatile uint32_t *polls, uint32_t rounds = 1) {
  const uint32_t bar = smem_u32(&barrier);
#pragma unroll 1
  for (uint32_t n = 1;; ++n) {
    const bool ok = tree_poll(bar, parity & 1u);
    if (__all_sync(0xffffffffu, ok)) return true;
    const bool stop = n >= *polls * rounds;
    if (__any_sync(0xffffffffu, stop)) break;
  }
  if (atomicExch(const_cast<uint32_t *>(polls), 0u) != 0) record_error(6 /* FP8Q_ERR_TIMEOUT */);
  return false;
}
// The calling warp's share of an arrival.
__device__ __forceinline__ void tree_arrive(const uint64_t &barrier) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&barrier));
}

// An arrival of every thread, once its cp.async copies so far are there.
__device__ __forceinline__ void tree_arrive_copies(const uint64_t &barrier) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&barrier))
               : "memory");
}

__device__ __forceinline__ void tree_ld(uint32_t taddr, uint32_t (&r)[16]) {
  tmem_ld_32x32b_x16(taddr, r);
  tmem_ld_wait(r);
}

// What the CTA's roles share.
constexpr int kTreePieces = 4;   // descriptors in the ring
struct TreeTile {                // for the V warps
  int32_t slot[kTreeN];          // cache rows of the tile's positions, -1 where there is none
  int32_t g;                     // kv head (-1: no more tiles)
  int32_t piece;                 // 2 (1 + index of the piece), 1 more where the tile lies in the context
};
struct TreeShared {
  uint64_t k_full[kTreeStages], k_free[kTreeStages], t_full[kTreeStages], t_free[kTreeStages];
  uint64_t piece_full[kTreePieces], piece_free[kTreePieces];
  uint64_t q_full, q_free, v_full[2], s_full[2], p_full[2], pv_done[2], drain;
  uint64_t valid[8];             // per tile (mod 8): the positions that exist, one bit each
  TreePiece piece[kTreePieces];
  TreeTile tile[kTreeStages];
  int start_b;
  int64_t start_off;
  int64_t warp_sum[kTreeThreads / 32];
  uint32_t tmem;
  uint32_t polls;                // of a wait at most; 0 once one has given up
  int nan_piece;                 // 1 + index of the last piece with a NaN code in V that was taken out
  float ml[4][32][2];
  float4 o[4][32][5];            // 16 columns, rows 80 bytes apart
};

// The next piece of the ring for the calling warp; false where there is none.
__device__ __forceinline__ bool tree_take(TreeShared &sh, uint32_t ip, TreePiece &pc,
                                          uint32_t rounds = 1) {
  const uint32_t i = ip % kTreePieces;
  pc.t = pc.t_end = 0;
  if (!tree_wait(sh.piece_full[i], ip / kTreePieces, &sh.polls, rounds)) return false;
  pc = sh.piece[i];
  tree_arrive(sh.piece_free[i]);
  return pc.t_end > 0;
}

// The dims of kv head g that are NaN in a value row seen by row (node i), among the positions behind the
// tiles that lie in the context and within [t, t_end), whose column within its tile lies in
// [c0, c0 + nc).  Runs only where a NaN code was taken out of V, over 17 tiles at most (1024 nodes): a
// walk over the whole context once took 0.33 us a position, and the waits of other roles have limits.
template <int D>
__device__ __noinline__ uint4 tree_nan_dims(const TreeAttnArgs &a, TreePiece c, int i, int c0,
                                            int nc) {
  uint32_t dims[4] = {};
  const int words = (a.max_nodes + 63) / 64;
  const int64_t *mrow = a.mask ? a.mask + (c.first + i) * a.ldm : nullptr;
  for (int tile = max(c.t, c.ctx / kTreeN); tile < c.t_end; ++tile) {
    const uint64_t bits = tree_bits(mrow, words, i, tile * kTreeN - c.ctx);
    for (int col = c0; col < c0 + nc; ++col) {
      const int pos = tile * kTreeN + col;
      if (!((bits >> col) & 1) || pos >= c.ctx + c.n) continue;
      const int32_t blk = a.block_table[c.b * a.max_blocks + a.by_block(pos)];
      if (blk < 0 || blk >= a.num_blocks) continue;
      const int64_t slot = static_cast<int64_t>(blk) * a.block_size + pos % a.block_size;
      const uint4 *v = reinterpret_cast<const uint4 *>(a.v_cache + (slot * a.Hkv + c.g) * D);
      for (int w = 0; w < D / 32; ++w)
#pragma unroll 1
        for (int x = 0; x < 2; ++x) {
          const uint4 q = v[2 * w + x];
          const uint32_t word[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            // 0x80 where a byte is NaN; its four flags side by side
            const uint32_t m = ((word[y] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
            dims[w] |= ((m >> 7) * 0x10204080u >> 28) << (16 * x + 4 * y);
          }
        }
    }
  }
  return make_uint4(dims[0], dims[1], dims[2], dims[3]);
}

// One row tile's running state in a softmax thread.
struct TreeRow {
  float ref, l;                  // reference of the weights (log2 units), their sum
};

// One position tile: the scores of 16 * chunks columns of this thread's row become weights, in the
// first half of the score buffer's columns: 8 columns per chunk, behind those already read.  The first
// chunk's scores stay in registers between the maximum and the weights, the others are read again.
// Loops over short bodies: the roles' code together has to stay in the instruction caches.  j0: the
// tile's first position, counted from node 0.
template <int D>
__device__ __forceinline__ bool tree_tile(TreeShared &sh, uint32_t tmem, uint32_t col0, int chunks,
                                          uint32_t it, bool first, const int64_t *mrow, int words,
                                          int node, int j0, float c2, TreeRow &st) {
  using L = TreeLayout<D>;
  if (!tree_wait(sh.s_full[it & 1u], it >> 1, &sh.polls)) return false;
  tc_fence_after();
  const uint32_t buf = tmem + L::kColS + 64 * (it & 1u);
  uint32_t sr[16];
  uint64_t seen = sh.valid[it & 7u];
  if (j0 > -kTreeN || seen != ~0ull) {                           // not within the context, or not whole
    // what is not seen becomes -inf in TMEM; a row that does not exist counts as seeing all
    if (node >= 0) seen &= tree_bits(mrow, words, node, j0);
    seen >>= col0;
#pragma unroll 1
    for (int c = 0; c < 16 * chunks; c += 16, seen >>= 16) {
      __syncwarp();                                              // whole warps at the TMEM loads
      tree_ld(buf + col0 + c, sr);
      const uint32_t bits = static_cast<uint32_t>(seen);
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (!((bits >> j) & 1)) sr[j] = 0xFF800000u;
      __syncwarp();
      tmem_st_32x32b_x16(buf + col0 + c, sr);
    }
    tmem_st_wait();
  }
  float mx[2] = {-INFINITY, -INFINITY};
  int c = chunks;
#pragma unroll 1
  do {
    --c;
    tree_ld(buf + col0 + 16 * c, sr);
#pragma unroll
    for (int j = 0; j < 16; ++j) mx[j & 1] = fmaxf(mx[j & 1], __uint_as_float(sr[j]));
  } while (c > 0);
  const float top = fmaxf(mx[0], mx[1]) * c2;
  const bool up = top > st.ref + kTreeLag;                       // also the first score seen
  if (__any_sync(0xffffffffu, up)) {
    const bool held = up && st.ref != -INFINITY;                 // values to rescale
    const float f = up ? tree_ex2(st.ref - top) : 1.0f;          // 0 from -inf
    st.ref = up ? top : st.ref;
    st.l *= f;
    if (!first && __any_sync(0xffffffffu, held)) {
      if (!tree_wait(sh.pv_done[(it - 1) & 1u], (it - 1) >> 1, &sh.polls)) return false;
      tc_fence_after();
#pragma unroll 1
      for (int d = 0; d < D; d += 16) {
        uint32_t o[16];
        tree_ld(tmem + L::kColO + d, o);
#pragma unroll
        for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
        tmem_st_32x32b_x16(tmem + L::kColO + d, o);
      }
    }
  }
  const float bias = kTreeBias - (st.ref == -INFINITY ? 0.0f : st.ref);
  const float2 c22 = make_float2(c2, c2), bias2 = make_float2(bias, bias);
  float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll 1
  while (true) {
    uint32_t pk[8];
#pragma unroll
    for (int j = 0; j < 16; j += 2) {
      const float2 z = f2_fma_rn(make_float2(__uint_as_float(sr[j]), __uint_as_float(sr[j + 1])), c22,
                                 bias2);
      const float2 w = make_float2(tree_ex2(z.x), tree_ex2(z.y));
      sum = f2_add_rn(sum, w);
      pk[j / 2] = f32x2_to_f16x2(w.x, w.y);
    }
    tmem_st_32x32b_x8(buf + col0 / 2 + 8 * c, pk);
    if (++c >= chunks) break;
    tree_ld(buf + col0 + 16 * c, sr);
  }
  // a repeat of a row has no weight at the other repeats' positions
#pragma unroll 1
  for (int i = 8 * chunks; i < 32; i += 8) {
    const uint32_t z[8] = {};
    tmem_st_32x32b_x8(buf + ((col0 / 2 + i) & 31u), z);
  }
  st.l += sum.x + sum.y;
  tmem_st_wait();
  tc_fence_before();
  tree_arrive(sh.p_full[it & 1u]);
  return true;
}

// Barrier of the four softmax warps, and one that tells whether any of them gave up.  Their waits are
// bounded and every one of them passes the same barriers.
__device__ __forceinline__ void tree_sync4() {
  __syncwarp();
  asm volatile("bar.sync 1, 128;" ::: "memory");
}
__device__ __forceinline__ bool tree_any4(bool v) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(v))
      : "memory");
  return r != 0;
}

template <int D>
__global__ void __launch_bounds__(kTreeThreads, 2)
    k_tree_attn(const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ TreeAttnArgs a) {
  using L = TreeLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ TreeShared sh;
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.Hq / a.Hkv;

  if (tid == 0) {
    for (int i = 0; i < kTreeStages; ++i) {
      mbar_init(smem_u32(&sh.k_full[i]), L::by_row(a.box) ? 33 : 1);   // its lanes and lane 0
      mbar_init(smem_u32(&sh.k_free[i]), 1);
      mbar_init(smem_u32(&sh.t_full[i]), 1);
      mbar_init(smem_u32(&sh.t_free[i]), 2);
    }
    for (int i = 0; i < kTreePieces; ++i) {
      mbar_init(smem_u32(&sh.piece_full[i]), 1);
      mbar_init(smem_u32(&sh.piece_free[i]), 6);
    }
    mbar_init(smem_u32(&sh.q_full), 1);
    mbar_init(smem_u32(&sh.q_free), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sh.v_full[i]), 2);
      mbar_init(smem_u32(&sh.p_full[i]), 4);
      mbar_init(smem_u32(&sh.pv_done[i]), 1);
      mbar_init(smem_u32(&sh.s_full[i]), 1);
    }
    mbar_init(smem_u32(&sh.drain), 1);
    sh.polls = a.polls;
    sh.nan_piece = 0;
    fence_barrier_init();
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
      mine += tree_group_cost(a, tree_seq(a, b, blockIdx.x == 0), G) * a.Hkv;
    }
    upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += y;
    }
    if (lane == 31) sh.warp_sum[warp] = upto;
    __syncwarp();                                                // whole warps at every barrier
    if (!__syncthreads_or(falls) || again) break;
    if (tid == 0) sh.start_b = a.B;
    __syncthreads();
    for (int b = tid * per; b < min(B, (tid + 1) * per); ++b)
      if (a.cu[b + 1] < a.cu[b]) {
        atomicMin(&sh.start_b, b);
        break;
      }
    __syncwarp();
    __syncthreads();
    B = sh.start_b;
    __syncthreads();
  }
  total = 0;
  for (int w = 0; w < kTreeThreads / 32; ++w) {
    if (w < warp) upto += sh.warp_sum[w];
    total += sh.warp_sum[w];
  }
  // an even share, at least kTreeMinCost (the last CTAs may have less, or nothing)
  const int64_t share = max(static_cast<int64_t>(kTreeMinCost),
                            static_cast<int64_t>(__umul64hi(total, a.grid_recip)) + 1);
  const int64_t lo = min(total, share * blockIdx.x), hi = min(total, lo + share);
  const bool works = lo < hi;
  int32_t *meta = a.meta + blockIdx.x * kTreeMetaInts;
  if (tid == 0) meta[0] = meta[1] = 0;
  if (works && lo >= upto - mine && lo < upto) {
    int64_t off = lo - (upto - mine);
    int b = tid * per;
    for (;; ++b) {
      const int64_t c = tree_group_cost(a, tree_seq(a, b, false), G) * a.Hkv;
      if (off < c) break;
      off -= c;
    }
    sh.start_b = b;
    sh.start_off = off;
  }
  __syncwarp();
  // only now that every warp of the CTA has started
  if (warp == 8) {
    tmem_alloc(smem_u32(&sh.tmem), L::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;

  if (warp == 9) {
    // ---------------------------------------------------------------- load
    // A copy brings `box` consecutive positions of one block; lane i holds the slot of the i-th copy's
    // first.  Where a copy would be small, rows go by cp.async; then lane i holds the slots of the
    // positions i and i + 32.
    TreeCursor pre;
    pre.init(a, G, B, sh.start_b, sh.start_off, hi - lo);
    const bool by_row = L::by_row(a.box);
    const int chunks = kTreeN / a.box, log_box = __ffs(a.box) - 1;
    const int first = by_row ? lane : min(lane, chunks - 1) * a.box;
    int blk[2], off[2];
    auto look_up = [&]() {                                       // block ids of the cursor's tile
      if (!pre.live) return;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (j == 1 && !by_row) break;
        const int pos = pre.t * kTreeN + 32 * j + first;
        const int q = a.by_block(pos);
        off[j] = pos - q * a.block_size;
        blk[j] = -1;
        if (pos < pre.s.ctx + pre.s.n) blk[j] = a.block_table[pre.b * a.max_blocks + q];
        else off[j] = -1;                                        // behind the sequence
      }
    };
    auto slot_of = [&](int j, bool *ok) {                        // row 0 for a place not seen
      *ok = blk[j] >= 0 && blk[j] < a.num_blocks;
      if (!*ok && off[j] >= 0) record_error(9 /* FP8Q_ERR_RANGE */);
      return *ok ? blk[j] * a.block_size + off[j] : 0;
    };
    uint32_t ip = 0;
    auto publish = [&]() {                                       // the piece, or the end
      const uint32_t i = ip % kTreePieces;
      if (!tree_wait(sh.piece_free[i], (ip / kTreePieces) ^ 1u, &sh.polls)) return false;
      if (lane == 0)
        sh.piece[i] = TreePiece{pre.s.first, pre.b, pre.s.n, pre.s.ctx, pre.g, pre.rt * kTreeM,
                                min(kTreeM, pre.s.n * G - pre.rt * kTreeM), pre.t,
                                pre.live ? pre.t_end : 0, pre.nt};
      tree_arrive(sh.piece_full[i]);
      ++ip;
      return true;
    };
    look_up();
    uint32_t it = 0, st = 0, ph = 1u;
    bool fresh = true;
    for (;; ++it) {
      if (fresh && !publish()) break;
      if (!pre.live) break;
      // the stage first: the block ids are on their way meanwhile
      if (!tree_wait(sh.k_free[st], ph, &sh.polls) ||
          !tree_wait(sh.t_free[st], ph, &sh.polls))
        break;
      bool ok;
      int32_t slot[2] = {slot_of(0, &ok), 0};
      uint64_t there;
      if (by_row) {
        there = __ballot_sync(0xffffffffu, ok);
        slot[1] = slot_of(1, &ok);
        there |= static_cast<uint64_t>(__ballot_sync(0xffffffffu, ok)) << 32;
      } else {
        const int left = pre.s.ctx + pre.s.n - pre.t * kTreeN;   // positions that exist
        there = ~0ull;
        if (left < 64 || !__all_sync(0xffffffffu, ok)) {
          const uint64_t bits = ok ? (a.box == 64 ? ~0ull : ((1ull << a.box) - 1) << first) : 0ull;
          there = __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(bits));
          there |= static_cast<uint64_t>(
                       __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(bits >> 32))) << 32;
          if (left < 64) there &= (1ull << left) - 1;
        }
      }
      const uint32_t bar = smem_u32(&sh.k_full[st]);
      if (lane == 0) {
        sh.valid[it & 7u] = there;
        sh.tile[st].g = pre.g;
        sh.tile[st].piece = static_cast<int>(2 * ip) + (pre.s.ctx >= (pre.t + 1) * kTreeN);
        if (by_row) mbar_arrive(bar);
        else mbar_arrive_expect_tx(bar, L::kTile);
      }
      __syncwarp();
      const uint32_t dst = sbase + L::kK + st * L::kTile;
      if (by_row) {
        constexpr int LPR = D / 16, RPS = 32 / LPR;              // lanes per row, rows per step
        const int ch = lane % LPR;
        const uint8_t *src = a.k_cache + pre.g * D + ch * 16;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll 4
          for (int r = lane / LPR; r < 32; r += RPS) {
            const int64_t from = __shfl_sync(0xffffffffu, slot[j], r);
            const int to = 32 * j + r, x = D == 128 ? to & 7 : to >> 1 & 3;
            cp_async16(dst + to * D + ((ch ^ x) << 4), src + from * a.Hkv * D,
                       (there >> to) & 1u ? 16u : 0u);
          }
        }
        tree_arrive_copies(sh.k_full[st]);
      } else {
        if (lane < chunks) tma_load_2d(dst + lane * a.box * D, &tm_k, pre.g * D, slot[0], bar);
        const int32_t row = slot[0];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int p = 32 * j + lane;
          slot[j] = __shfl_sync(0xffffffffu, row, p >> log_box) + (p & (a.box - 1));
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j)
        sh.tile[st].slot[32 * j + lane] = (there >> (32 * j + lane)) & 1u ? slot[j] : -1;
      tree_arrive(sh.t_full[st]);
      if (++st == kTreeStages) {
        st = 0;
        ph ^= 1u;
      }
      fresh = ++pre.t >= pre.t_end;
      if (fresh) pre.next(a, G, 0);
      look_up();
    }
    // the end, for both pairs of V warps
    for (int i = 0; i < 2; ++i) {
      if (!tree_wait(sh.t_free[st], ph, &sh.polls)) break;
      if (lane == 0) sh.tile[st].g = -1;
      tree_arrive(sh.t_full[st]);
      if (++st == kTreeStages) {
        st = 0;
        ph ^= 1u;
      }
    }
    // after a wait that gave up: no copy in flight at exit
    for (uint32_t i = it < kTreeStages ? 0 : it - kTreeStages; i < it; ++i)
      wait_drain(smem_u32(&sh.k_full[i % kTreeStages]), i / kTreeStages & 1u);
  } else if (warp == 10) {
    // ---------------------------------------------------------------- queries
    constexpr int LPR = D / 16;                                  // 16-byte chunks per row
    const float c = a.sm_scale * a.scale3[0] * a.scale3[1];
    const uint32_t qflip = c < 0.0f ? 0x80808080u : 0u;          // a negative scale negates Q
    // The next piece is not published before the load warp has come through this one: a wait of as many
    // tiles (at most 2^32 polls).  Without it pieces that took longer than the limit, 40 million
    // positions and more, were given up.
    TreePiece pc;
    bool ok = true;
    uint32_t rounds = 1;
    for (uint32_t ip = 0; ok && tree_take(sh, ip, pc, rounds); ++ip) {
      rounds = min(pc.t_end - pc.t + 1, (1 << 14) - 1);
      // Row r is head g G + r % G of node r / G; up to 32 (64) rows are repeated 4 (2) times down the
      // tile.  The first 256 chunks are on their way while the scores of the piece before complete,
      // the others all at once behind them.
      const int step = pc.rows <= 32 ? 32 : (pc.rows <= 64 ? 64 : 128);
      auto source = [&](int r) {
        const int idx = pc.row0 + r, node = a.by_group(idx), h = pc.g * G + (idx - node * G);
        return a.q + (pc.first + node) * a.ldq + h * D;
      };
      uint4 v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int i = 32 * k + lane, r = i / LPR;
        v[k] = make_uint4(0, 0, 0, 0);
        if (r < min(pc.rows, step))
          v[k] = *reinterpret_cast<const uint4 *>(source(r) + i % LPR * 16);
      }
      if (!(ok = tree_wait(sh.q_free, ip ^ 1u, &sh.polls))) break;
#pragma unroll 1
      for (int i = 256 + lane; i < step * LPR; i += 32) {
        const int r = i / LPR, x = (i % LPR ^ (r & 7)) << 4;
        const uint8_t *src = source(min(r, pc.rows - 1)) + i % LPR * 16;
        for (int rr = r; rr < kTreeM; rr += step)
          cp_async16(sbase + L::kQ + rr * 128 + x, src, r < pc.rows ? 16u : 0u);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int i = 32 * k + lane, r = i / LPR;
        v[k].x ^= qflip; v[k].y ^= qflip; v[k].z ^= qflip; v[k].w ^= qflip;
        for (int rr = r; r < step && rr < kTreeM; rr += step)
          *reinterpret_cast<uint4 *>(smem + L::kQ + rr * 128 + ((i % LPR ^ (r & 7)) << 4)) = v[k];
      }
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      if (qflip != 0) {
#pragma unroll 1
        for (int i = 256 + lane; i < step * LPR; i += 32) {
          const int r = i / LPR, x = (i % LPR ^ (r & 7)) << 4;
          for (int rr = r; rr < kTreeM; rr += step) {
            uint4 *q = reinterpret_cast<uint4 *>(smem + L::kQ + rr * 128 + x);
            *q = make_uint4(q->x ^ qflip, q->y ^ qflip, q->z ^ qflip, q->w ^ qflip);
          }
        }
      }
      fence_proxy_async_shared();
      tree_arrive(sh.q_full);
    }
  } else if (warp >= 4 && warp < 8) {
    // ---------------------------------------------------------------- V codes to fp16
    // Two pairs of warps take the tiles in turn, each into its own buffer.
    constexpr int LPR = D / 16;                                  // lanes per row
    constexpr int RPS = 64 / LPR, NR = kTreeN / RPS;             // rows per step, steps
    // a quarter warp's 16-byte stores cover all banks: its lanes hold four chunks of one half of two
    // neighbouring rows
    const int pair = (warp - 4) >> 1, gt = tid - 128 - 64 * pair;
    const int ch = D == 128 ? (gt & 3) | (gt >> 1 & 4) : gt & 3;
    const int r0 = D == 128 ? (gt >> 2 & 1) | (gt >> 4 << 1) : gt >> 2;
    const int64_t row = static_cast<int64_t>(a.Hkv) * D;
    const uint32_t stage = sbase + L::kV8 + pair * L::kTile + gt * 16;
    for (uint32_t it = pair;; it += 2) {
      const uint32_t st = it % kTreeStages;
      if (!tree_wait(sh.t_full[st], it / kTreeStages, &sh.polls)) break;
      const TreeTile &tile = sh.tile[st];
      const int32_t g = tile.g, piece = tile.piece;
      if (g < 0) break;
      // each thread copies and converts 16 codes of every step's row
      const uint8_t *col = a.v_cache + g * D + ch * 16;
#pragma unroll 2
      for (int j = 0; j < NR; ++j) {
        const int32_t slot = tile.slot[j * RPS + r0];
        cp_async16(stage + j * 1024, col + static_cast<int64_t>(max(slot, 0)) * row,
                   slot >= 0 ? 16u : 0u);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      tree_arrive(sh.t_free[st]);
      if (it >= 2 && !tree_wait(sh.pv_done[pair], (it - 2) >> 1, &sh.polls)) break;
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      uint8_t *dst = smem + L::kV16 + pair * L::kV16Bytes + (ch >> 2) * 8192 + r0 * 128;
      const int at0 = ((ch & 3) * 2 ^ (r0 & 7)) << 4;            // RPS is a multiple of 8
#pragma unroll 1
      for (int j = 0; j < NR; j += 2) {
        uint4 v8[2];
        uint32_t h[16];
#pragma unroll
        for (int k = 0; k < 2; ++k)
          v8[k] = *reinterpret_cast<const uint4 *>(smem + (stage - sbase) + (j + k) * 1024);
        while (true) {
          const uint32_t w[8] = {v8[0].x, v8[0].y, v8[0].z, v8[0].w,
                                 v8[1].x, v8[1].y, v8[1].z, v8[1].w};
          __half2 m[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            h[2 * k] = e4m3x2_to_f16x2(w[k] & 0xFFFFu);
            h[2 * k + 1] = e4m3x2_to_f16x2(w[k] >> 16);
            m[k] = __hmax2_nan(*reinterpret_cast<const __half2 *>(&h[2 * k]),
                               *reinterpret_cast<const __half2 *>(&h[2 * k + 1]));
          }
#pragma unroll
          for (int d = 4; d > 0; d /= 2)
#pragma unroll
            for (int k = 0; k < d; ++k) m[k] = __hmax2_nan(m[k], m[k + d]);
          if (!__hisnan(__low2half(m[0])) && !__hisnan(__high2half(m[0]))) break;
          // A NaN code of a tile in the context stays: every row sees it, and the products bring it to
          // them.  Else, where some rows may not see it, it becomes 0 and is put back into the results
          // of the rows that do.
          if (piece & 1) break;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t *x[4] = {&v8[k].x, &v8[k].y, &v8[k].z, &v8[k].w};
#pragma unroll
            for (int q = 0; q < 4; ++q)
              *x[q] &= ~(((((*x[q] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7) * 0xFFu);
          }
          atomicMax(&sh.nan_piece, piece >> 1);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint8_t *d = dst + (j + k) * RPS * 128;
          *reinterpret_cast<uint4 *>(d + at0) =
              make_uint4(h[8 * k], h[8 * k + 1], h[8 * k + 2], h[8 * k + 3]);
          *reinterpret_cast<uint4 *>(d + (at0 ^ 16)) =
              make_uint4(h[8 * k + 4], h[8 * k + 5], h[8 * k + 6], h[8 * k + 7]);
        }
      }
      fence_proxy_async_shared();
      tree_arrive(sh.v_full[pair]);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");         // none in flight at exit
  } else if (warp == 8) {
    // ---------------------------------------------------------------- MMA issue
    // The whole warp runs the loop, so that addresses stay in uniform registers; one lane issues.
    {
      const bool leader = elect_one();
      const uint64_t qd = tree_sdesc_k<128>(sbase + L::kQ);
      uint32_t ip = 0;
      int left = 0;
      bool fresh = false, before = false;
      auto next = [&]() {                                        // the next tile, if there is one
        fresh = left == 0;
        if (fresh) {
          const uint32_t i = ip % kTreePieces;
          if (!tree_wait(sh.piece_full[i], ip / kTreePieces, &sh.polls)) return false;
          left = sh.piece[i].t_end - (sh.piece[i].t_end > 0 ? sh.piece[i].t : 0);
          tree_arrive(sh.piece_free[i]);
          ++ip;
        }
        return left-- > 0;
      };
      uint32_t st = 0, ph = 0;
      bool live = next();
      // the scores of tile it, then the values of tile it - 1
#pragma unroll 1
      for (uint32_t it = 0;; ++it) {
        // The scores' buffer held the weights of tile it - 2, which the MMAs issued before read.  The
        // values come first where the scores wait for another piece's queries.
        bool ok = true;
#pragma unroll 1
        for (int k = 0; k < 2 && ok; ++k) {
          if (fresh == (k == 1)) {
            if (!live) continue;
            if ((fresh && !tree_wait(sh.q_full, ip - 1, &sh.polls)) ||
                !tree_wait(sh.k_full[st], ph, &sh.polls)) {
              ok = false;
              continue;
            }
            if (L::by_row(a.box)) fence_proxy_async_shared();    // K came by cp.async
            tc_fence_after();
            const uint64_t kd = tree_sdesc_k<D>(sbase + L::kK + st * L::kTile);
            if (leader) {
#pragma unroll
              for (int kk = 0; kk < D / 32; ++kk)
                mma_f8f6f4(tmem + L::kColS + 64 * (it & 1u), qd + 2 * kk, kd + 2 * kk, L::kIdescQK,
                           kk > 0 ? 1u : 0u);
              mma_commit(smem_u32(&sh.s_full[it & 1u]));
              mma_commit(smem_u32(&sh.k_free[st]));
              if (left == 0) mma_commit(smem_u32(&sh.q_free));   // the piece's last scores
            }
            __syncwarp();
            if (++st == kTreeStages) {
              st = 0;
              ph ^= 1u;
            }
          } else if (it > 0) {
            const uint32_t i = (it - 1) & 1u, pp = (it - 1) >> 1;
            if (!tree_wait(sh.p_full[i], pp, &sh.polls) ||
                !tree_wait(sh.v_full[i], pp, &sh.polls)) {
              ok = false;
              continue;
            }
            tc_fence_after();
            const uint64_t vd = tree_sdesc_v(sbase + L::kV16 + i * L::kV16Bytes);
            if (leader) {
#pragma unroll
              for (int kk = 0; kk < kTreeN / 16; ++kk)
                mma_f16_ts(tmem + L::kColO, tmem + L::kColS + 64 * i + 8 * kk, vd + 128 * kk,
                           L::kIdescPV, before && kk == 0 ? 0u : 1u);
              mma_commit(smem_u32(&sh.pv_done[i]));
            }
            __syncwarp();
          }
        }
        if (!ok) break;
        if (!live) break;
        before = fresh;
        live = next();
      }
      if (leader) mma_commit(smem_u32(&sh.drain));               // all MMAs done before dealloc
      __syncwarp();
      wait_drain(smem_u32(&sh.drain), 0);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- softmax and output
    float c2 = fabsf(a.sm_scale * a.scale3[0] * a.scale3[1]) * 1.4426950408889634f;
    c2 = c2 < 1e-37f ? 1e-37f : c2;                              // so that -inf stays -inf
    const float sv = a.scale3[2];
    const uint32_t tw = tmem + (static_cast<uint32_t>(32 * warp) << 16);
    const int words = (a.max_nodes + 63) / 64;
    uint32_t it = 0;
    TreePiece pc;
    for (uint32_t ip = 0;; ++ip) {
      bool ok = tree_take(sh, ip, pc);
      const int shift = pc.rows <= 32 ? 2 : (pc.rows <= 64 ? 1 : 0), rep = 1 << shift;
      const int w0 = warp & ((4 >> shift) - 1), r = 32 * w0 + lane, nc = kTreeN >> shift;
      const uint32_t col0 = nc * (warp >> (2 - shift));
      const bool live = r < pc.rows;
      const int node = a.by_group(pc.row0 + r);
      const int64_t *mrow = a.mask && live ? a.mask + (pc.first + node) * a.ldm : nullptr;
      TreeRow st{-INFINITY, 0.0f};
      for (int t = pc.t; t < pc.t_end && ok; ++t, ++it) {
        ok = tree_tile<D>(sh, tw, col0, 4 >> shift, it, t == pc.t, mrow, words, live ? node : -1,
                          t * kTreeN - pc.ctx, c2, st);
      }
      ok = ok && tree_wait(sh.pv_done[(it - 1) & 1u], (it - 1) >> 1, &sh.polls);
      sh.ml[warp][lane][0] = st.ref;
      sh.ml[warp][lane][1] = st.l;
      if (tree_any4(!ok)) break;                                 // no more pieces, or given up
      tc_fence_after();
      uint4 nan = make_uint4(0, 0, 0, 0);
      const bool any_nan = *reinterpret_cast<volatile int *>(&sh.nan_piece) > static_cast<int>(ip);
      if (any_nan && live) nan = tree_nan_dims<D>(a, pc, node, col0, nc);
      const bool whole = pc.t == 0 && pc.t_end == pc.nt;
      const int slot = pc.t > 0 ? 0 : 1;
      float *part = a.part + (static_cast<int64_t>(blockIdx.x) * 2 + slot) * a.row_cap * (D + 2);
      if (tid == 0 && !whole) {
        if (slot == 0) meta[0] = pc.t_end == pc.nt ? 2 : 1;      // a part; 2: the item's last
        else {
          meta[1] = 1;                                           // the item's first part
          meta[2] = static_cast<int>(pc.first);
          meta[3] = pc.row0;
          meta[4] = pc.rows;
          meta[5] = pc.g;
        }
      }
      // Repeats of a row hold different positions: their states are merged, then summed by rows, `rep`
      // threads per row and 16 / rep columns each.
      auto merged = [&](int w, int ln, float &l) {
        float M = -INFINITY;
        for (int i = w; i < 4; i += 4 >> shift) M = fmaxf(M, sh.ml[i][ln][0]);
        l = 0.0f;
        for (int i = w; i < 4; i += 4 >> shift) {
          const float m = sh.ml[i][ln][0];
          l += sh.ml[i][ln][1] * (m == M ? 1.0f : tree_ex2(m - M));
        }
        return M;
      };
      const int tr = tid >> shift, cpt = 16 >> shift, tc = (tid & (rep - 1)) * cpt;
      float l;
      const float mine_M = merged(w0, lane, l);
      const float f = st.l == 0.0f ? 0.0f : (st.ref == mine_M ? 1.0f : tree_ex2(st.ref - mine_M));
      const float M = merged(tr >> 5, tr & 31, l);
      const float scale = whole ? (l == 0.0f ? 0.0f : sv / l) : 1.0f;
      const int idx = pc.row0 + tr, nd = a.by_group(idx), h = pc.g * G + (idx - nd * G);
      uint16_t *out = a.out + (pc.first + nd) * a.ldo + h * D + tc;
      float *po = part + tr * D + tc;
      auto store4 = [&](int c, float4 v) {
        if (whole) {
          const __nv_bfloat162 b0 = __floats2bfloat162_rn(v.x * scale, v.y * scale);
          const __nv_bfloat162 b1 = __floats2bfloat162_rn(v.z * scale, v.w * scale);
          *reinterpret_cast<uint2 *>(out + c) =
              make_uint2(*reinterpret_cast<const uint32_t *>(&b0),
                         *reinterpret_cast<const uint32_t *>(&b1));
        } else {
          *reinterpret_cast<float4 *>(po + c) = v;
        }
      };
#pragma unroll 1
      for (int c = 0; c < D; c += 16) {
        uint32_t o[16];
        __syncwarp();
        tree_ld(tw + L::kColO + c, o);
        float4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          v[j] = make_float4(__uint_as_float(o[4 * j]) * f, __uint_as_float(o[4 * j + 1]) * f,
                             __uint_as_float(o[4 * j + 2]) * f, __uint_as_float(o[4 * j + 3]) * f);
        if (any_nan) {
          const uint32_t w = (c < 64 ? (c < 32 ? nan.x : nan.y) : (c < 96 ? nan.z : nan.w)) >> (c & 31);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if ((w >> (4 * j)) & 1u) v[j].x = NAN;
            if ((w >> (4 * j)) & 2u) v[j].y = NAN;
            if ((w >> (4 * j)) & 4u) v[j].z = NAN;
            if ((w >> (4 * j)) & 8u) v[j].w = NAN;
          }
        }
        if (rep == 1) {
          if (live) {
#pragma unroll
            for (int j = 0; j < 4; ++j) store4(c + 4 * j, v[j]);
          }
          continue;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) sh.o[warp][lane][j] = v[j];
        tree_sync4();
        if (tr < pc.rows) {
          // four reads: four warps' columns, or two warps' twice as many
          float4 x[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            x[j] = rep == 4 ? sh.o[j][tr][tid & 3]
                            : sh.o[(tr >> 5) + 2 * (j & 1)][tr & 31][2 * (tid & 1) + (j >> 1)];
          const float4 s0 = make_float4(x[0].x + x[1].x, x[0].y + x[1].y, x[0].z + x[1].z,
                                        x[0].w + x[1].w);
          const float4 s1 = make_float4(x[2].x + x[3].x, x[2].y + x[3].y, x[2].z + x[3].z,
                                        x[2].w + x[3].w);
          if (rep == 4) {
            store4(c, make_float4(s0.x + s1.x, s0.y + s1.y, s0.z + s1.z, s0.w + s1.w));
          } else {
            store4(c, s0);
            store4(c + 4, s1);
          }
        }
        tree_sync4();
      }
      if (!whole && tr < pc.rows && tc == 0) {
        float *ml = part + static_cast<int64_t>(a.row_cap) * D;
        ml[2 * tr] = M;
        ml[2 * tr + 1] = l;
      }
      tc_fence_before();
    }
  }

  __syncwarp();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    __syncwarp();
    tmem_dealloc(tmem, L::kCols);
  }
}

// The items that several CTAs shared: block (i, y) takes the rows 8 y .. 8 y + 7 of the item whose
// first part is CTA i's last piece, a warp per row, and adds the parts in CTA order, each a running
// maximum's state.
template <int D>
__global__ void __launch_bounds__(256) k_tree_attn_combine(const TreeAttnArgs a) {
  constexpr int V = D / 32;
  static_assert(V == 2 || V == 4, "vector loads of the parts");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int i = blockIdx.x, lane = threadIdx.x & 31;
  const int32_t *meta = a.meta + i * kTreeMetaInts;
  const int4 m0 = *reinterpret_cast<const int4 *>(meta);         // part, first part, row of node 0, row0
  const int2 m1 = *reinterpret_cast<const int2 *>(meta + 4);     // rows, kv head
  const int r = blockIdx.y * 8 + (threadIdx.x >> 5);
  if (m0.y == 0 || r >= m1.x) return;
  const int64_t slot = static_cast<int64_t>(a.row_cap) * (D + 2);
  const float *base = a.part + r * D + V * lane;
  const int64_t ml = static_cast<int64_t>(a.row_cap) * D + 2 * r;
  float top = -INFINITY, l = 0.0f, o[V] = {};
  // 32 parts at a time: their maxima and sums by lanes, then the values one after the other
  for (int j0 = i;; j0 += 32) {
    const int j = j0 + lane;
    const bool in = j < static_cast<int>(gridDim.x);
    const int kind = j == i ? 1 : (in ? a.meta[j * kTreeMetaInts] : 2);
    const uint32_t ends = __ballot_sync(0xffffffffu, kind != 1);
    const int last = ends ? __ffs(ends) - 1 : 31;
    const int n = __shfl_sync(0xffffffffu, last + (in ? 1 : 0), last);  // behind the grid: not a part
    float2 e = make_float2(-INFINITY, 0.0f);                     // maximum, sum
    if (lane < n)
      e = *reinterpret_cast<const float2 *>(
          a.part + (2 * static_cast<int64_t>(j) + (j == i ? 1 : 0)) * slot + ml);
    if (e.y == 0.0f) e.x = -INFINITY;
    float m = e.x;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    m = fmaxf(m, top);
    // a part without weight has l = 0; a NaN sum stays one
    const float w = e.y == 0.0f ? 0.0f : (e.x == m ? 1.0f : tree_ex2(e.x - m));
    const float keep = l == 0.0f ? 0.0f : (top == m ? 1.0f : tree_ex2(top - m));
    float sum = e.y * w;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    l = l * keep + sum;
    top = m;
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] *= keep;
#pragma unroll 2
    for (int k = 0; k < n; ++k) {
      const float *p = base + (2 * static_cast<int64_t>(j0 + k) + (j0 + k == i ? 1 : 0)) * slot;
      const float wk = __shfl_sync(0xffffffffu, w, k);
      alignas(16) float v[V];
      if constexpr (V == 4) *reinterpret_cast<float4 *>(v) = *reinterpret_cast<const float4 *>(p);
      else *reinterpret_cast<float2 *>(v) = *reinterpret_cast<const float2 *>(p);
#pragma unroll
      for (int x = 0; x < V; ++x) o[x] += v[x] * wk;
    }
    if (ends) break;
  }
  const int G = a.Hq / a.Hkv, idx = m0.w + r, node = a.by_group(idx);
  const int h = m1.y * G + (idx - node * G);
  const float f = l == 0.0f ? 0.0f : a.scale3[2] / l;
  uint16_t *out = a.out + (static_cast<int64_t>(m0.z) + node) * a.ldo + h * D + V * lane;
#pragma unroll
  for (int v = 0; v < V; v += 2) {
    const __nv_bfloat162 b2 = __floats2bfloat162_rn(l == 0.0f ? 0.0f : o[v] * f,
                                                    l == 0.0f ? 0.0f : o[v + 1] * f);
    *reinterpret_cast<uint32_t *>(out + v) = *reinterpret_cast<const uint32_t *>(&b2);
  }
}

}  // namespace fp8q
