// spec_kernels.cuh -- the integer and data-movement operators of a speculative-decoding step over
// the paged FP8 KV cache, for sm_100a:
//   k_paged_tables   block tables, slot maps, positions and offsets from request lengths
//   k_tree_mask      ancestor bits and positions of drafted nodes from parent indices
//   k_kv_accept      rows of the accepted path moved to consecutive cache positions
// Inputs that break a rule record FP8Q_ERR_RANGE (9) in the device error word; what is read and
// written then stays inside the buffers, as each kernel states.
#pragma once
#include <cstdint>
#include "ptx.cuh"

namespace fp8q {

// ---------------------------------------------------------------------------------------------
// Block tables and slot maps
// ---------------------------------------------------------------------------------------------
constexpr int kTablesThreads = 512;
constexpr int kTablesMaxB = 16384;

struct TablesArgs {
  const int32_t *ctx_lens, *new_lens;  // [B]
  int B;
  uint32_t block_size;
  int32_t *block_table;                // [B][max_blocks]
  int64_t max_blocks;
  int64_t capacity;                    // max_blocks * block_size, at most INT32_MAX
  const int32_t *free_blocks;          // [num_free], a stack: the top is entry *free_count - 1
  int64_t num_free;
  const int32_t *free_count;
  int32_t *free_left;
  const int32_t *held;                 // [B] or null: blocks already held, beyond the context's too
  int32_t *held_out;                   // [B] or null
  int64_t max_tokens;
  int32_t *cu, *seq_lens;              // [B + 1], [B]
  int64_t *slots, *positions;          // [max_tokens]
};

// Exclusive prefix sum of v over the CTA; *total gets the sum.  s_warp: one word per warp.
__device__ __forceinline__ int64_t cta_exclusive_scan(int64_t v, int64_t *s_warp, int64_t *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();  // s_warp may still be read from the scan before
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  int64_t before = 0, all = 0;
  for (int w = 0; w < static_cast<int>(blockDim.x) / 32; ++w) {
    const int64_t s = s_warp[w];
    before += w < warp ? s : 0;
    all += s;
  }
  *total = all;
  return before + x - v;
}

// Blocks that request b holds: those of its c cached positions, and where the caller keeps count, those
// left from drafts whose nodes were rejected.
__device__ __forceinline__ uint32_t tables_have(const TablesArgs &a, int b, uint32_t c, bool *bad) {
  const uint32_t have = c / a.block_size + (c % a.block_size != 0);
  if (!a.held) return have;
  const int32_t h = a.held[b], most = static_cast<int32_t>(a.max_blocks);  // at most INT32_MAX
  *bad |= h < 0 || h > most;
  return max(have, static_cast<uint32_t>(max(0, min(h, most))));
}

// Request b has c = ctx_lens[b] cached positions in ceil(c / bs) blocks and adds n = new_lens[b]
// tokens at positions c .. c + n - 1, which reach into ceil((c + n) / bs) blocks; the blocks it
// lacks are popped from the free stack in request order.  With the prefix sums of n (tokens) and
// of the new blocks in shared memory every token finds its request by bisection, and its block
// either in the table (a block the request had) or in the stack; the first position of a new
// block is always a new token, so that token writes the table entry and no thread reads an entry
// that this launch writes.  Every CTA makes the prefix sums itself (2 B words from L2): one launch,
// no exchange between CTAs.  A decode step's 64 tokens take 4 us of device time (6 with nothing in L2),
// bound by the chain of dependent loads; a million tokens of 256 prompts 12 us (15), of it 2.6 for the
// bytes.
template <int R>
__global__ void __launch_bounds__(kTablesThreads) k_paged_tables(const TablesArgs a) {
  extern __shared__ int32_t s_tab[];          // [B + 1] token offsets, [B + 1] new-block offsets
  __shared__ int64_t s_warp[kTablesThreads / 32];
  int32_t *s_cu = s_tab, *s_nb = s_tab + a.B + 1;
  const int tid = threadIdx.x;
  const bool lead = blockIdx.x == 0;
  const uint32_t bs = a.block_size;
  bool bad = false;
  int64_t tokens = 0, blocks = 0;             // sums so far
  for (int base = 0; base < a.B; base += kTablesThreads) {
    const int b = base + tid;
    int64_t c = 0, n = 0;
    if (b < a.B) {
      const int32_t c0 = a.ctx_lens[b], n0 = a.new_lens[b];
      c = c0 < 0 ? 0 : (c0 > a.capacity ? a.capacity : c0);
      n = n0 < 0 ? 0 : n0;
      if (n > a.capacity - c) n = a.capacity - c;
      bad |= c != c0 || n != n0;
    }
    int64_t sum;
    const int64_t first = tokens + cta_exclusive_scan(n, s_warp, &sum);
    tokens += sum;
    const int64_t lo = first < a.max_tokens ? first : a.max_tokens;
    const int64_t hi = first + n < a.max_tokens ? first + n : a.max_tokens;
    bad |= hi != first + n;
    const int64_t have = b < a.B ? tables_have(a, b, static_cast<uint32_t>(c), &bad) : 0;
    const int64_t want = max(have, (c + (hi - lo) + bs - 1) / bs);
    const int64_t nb = blocks + cta_exclusive_scan(want - have, s_warp, &sum);
    blocks += sum;
    if (b < a.B) {
      s_cu[b] = static_cast<int32_t>(lo);
      s_nb[b] = static_cast<int32_t>(nb);
      if (lead) {
        a.cu[b] = static_cast<int32_t>(lo);
        a.seq_lens[b] = static_cast<int32_t>(c + (hi - lo));
      }
    }
  }
  const int32_t total = static_cast<int32_t>(tokens < a.max_tokens ? tokens : a.max_tokens);
  int64_t avail = *a.free_count;
  if (avail < 0 || avail > a.num_free) {
    bad = true;
    avail = avail < 0 ? 0 : a.num_free;
  }
  if (tid == 0) {
    s_cu[a.B] = total;
    if (lead) {
      a.cu[a.B] = total;
      *a.free_left = static_cast<int32_t>(avail > blocks ? avail - blocks : 0);
      bad |= blocks > avail;
    }
  }
  if (lead && a.held_out) {
    // where the stack runs short a request gets its lower entries, and the later requests none
    if (tid == 0) s_nb[a.B] = static_cast<int32_t>(blocks);
    __syncthreads();
    for (int b = tid; b < a.B; b += kTablesThreads) {
      const int64_t c0 = a.ctx_lens[b], need = s_nb[b + 1] - s_nb[b], left = avail - s_nb[b];
      const uint32_t c = static_cast<uint32_t>(c0 < 0 ? 0 : (c0 > a.capacity ? a.capacity : c0));
      const int64_t got = left < 0 ? 0 : (left < need ? left : need);
      a.held_out[b] = static_cast<int32_t>(tables_have(a, b, c, &bad) + got);
    }
  }
  if (lead && bad) record_error(9 /* FP8Q_ERR_RANGE */);
  __syncthreads();
  // R consecutive tokens per thread: a bisection where the request changes, a block id where the block
  // changes, 16-byte stores where the arrays allow them.
  const bool wide = R > 1 && ((reinterpret_cast<uintptr_t>(a.slots) |
                      reinterpret_cast<uintptr_t>(a.positions)) & 15u) == 0;
  for (int64_t t0 = R * (static_cast<int64_t>(blockIdx.x) * kTablesThreads + tid);
       t0 < a.max_tokens; t0 += R * static_cast<int64_t>(gridDim.x) * kTablesThreads) {
    int64_t slot[R], position[R];
    int lo = 0;
    int64_t end = t0;                          // of the request: none yet
    uint32_t pos = 0, blk = 0, off = 0, have = 0;
    int32_t id = -1;
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const int64_t t = t0 + j;
      slot[j] = -1;                            // behind the last token: a slot no cache write uses
      position[j] = 0;
      if (t >= total) continue;
      bool fetch = false;
      if (t >= end) {
        int hi = a.B;                          // s_cu[lo] <= t < s_cu[hi]
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (s_cu[mid] <= t) lo = mid; else hi = mid;
        }
        end = s_cu[lo + 1];
        const int64_t c0 = a.ctx_lens[lo];
        const uint32_t c = static_cast<uint32_t>(c0 < 0 ? 0 : (c0 > a.capacity ? a.capacity : c0));
        pos = c + static_cast<uint32_t>(t - s_cu[lo]);
        blk = pos / bs;
        off = pos - blk * bs;
        have = tables_have(a, lo, c, &bad);
        fetch = true;
      } else {
        ++pos;
        if (++off == bs) {
          off = 0;
          ++blk;
          fetch = true;
        }
      }
      if (fetch) {
        int32_t *entry = a.block_table + lo * a.max_blocks + blk;
        if (blk < have) {
          id = *entry;
        } else {
          const int64_t k = static_cast<int64_t>(s_nb[lo]) + (blk - have);
          id = k < avail ? a.free_blocks[avail - 1 - k] : -1;
          if (off == 0) *entry = id;
        }
      }
      slot[j] = id < 0 ? -1 : static_cast<int64_t>(id) * bs + off;
      position[j] = pos;
    }
    if (wide && t0 + R <= a.max_tokens) {
#pragma unroll
      for (int j = 0; j + 1 < R; j += 2) {
        *reinterpret_cast<longlong2 *>(a.slots + t0 + j) = make_longlong2(slot[j], slot[j + 1]);
        *reinterpret_cast<longlong2 *>(a.positions + t0 + j) =
            make_longlong2(position[j], position[j + 1]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < R; ++j)
        if (t0 + j < a.max_tokens) {
          a.slots[t0 + j] = slot[j];
          a.positions[t0 + j] = position[j];
        }
    }
  }
}

// ---------------------------------------------------------------------------------------------
// Ancestor masks
// ---------------------------------------------------------------------------------------------
constexpr int kTreeMaxNodes = 1024;

struct TreeMaskArgs {
  const int32_t *parents;            // [total]
  const int32_t *cu;                 // [B + 1]
  const int32_t *ctx_lens;           // [B] or null
  int64_t total;
  int max_nodes;
  int64_t *mask;                     // [total][ldm]
  int64_t ldm;
  int64_t *positions;                // [total] or null
};

// The rows [first, first + n) of sequence b: cu clamped into [0, total], at most max_nodes.
__device__ __forceinline__ int tree_rows(const int32_t *cu, int b, int64_t total, int max_nodes,
                                         int64_t *first, bool *bad) {
  const int64_t lo0 = cu[b], hi0 = cu[b + 1];
  int64_t lo = lo0 < 0 ? 0 : (lo0 > total ? total : lo0);
  int64_t n = (hi0 < 0 ? 0 : (hi0 > total ? total : hi0)) - lo;
  *bad = lo != lo0 || n != hi0 - lo0 || n < 0 || n > max_nodes;
  if (n < 0) n = 0;
  if (n > max_nodes) n = max_nodes;
  *first = lo;
  return static_cast<int>(n);
}

// One CTA per sequence and word of the rows: a word needs no other one.  Every CTA also looks through
// the offsets up to its sequence: where they decrease the batch ends, so that no two sequences write
// the same rows.  Pointer doubling: row i holds the nodes from i up to (not including) anc[i]; a
// round ORs in the row of anc[i] and jumps to anc[anc[i]], so a tree of depth d takes ceil(log2 d)
// rounds instead of d steps.  Word w needs no ancestor below its first node 64 w: anc is cut there.
// The first word's CTA counts the depths along the way.  Each round reads into registers, then
// writes, so no row is read while it changes.  16 trees of up to 1000 nodes take 8 us (one CTA per
// tree over all words took 80), 64 of up to 16 nodes 3 us: the rounds' latency.  The look through the
// offsets is quadratic in the batch: 15 us for 8000 sequences, 0.56 ms for 65535, and 10 ms with 16 words.
template <int T, int ITEMS>
__global__ void __launch_bounds__(T) k_tree_mask(const TreeMaskArgs a) {
  __shared__ uint64_t s_bits[T * ITEMS];
  __shared__ int32_t s_anc[T * ITEMS], s_depth[T * ITEMS];
  const int b = blockIdx.x, w = blockIdx.y, tid = threadIdx.x;
  int64_t first;
  bool bad, falls = false;
  const int n = tree_rows(a.cu, b, a.total, a.max_nodes, &first, &bad);
  for (int i = tid; i <= b; i += T) falls |= a.cu[i + 1] < a.cu[i];
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    const int i = tid + k * T;
    if (i >= n) continue;
    int p = a.parents[first + i];
    if (p < -1 || p >= i) {                                    // parents come first
      bad = true;
      p = -1;
    }
    s_anc[i] = p >= 64 * w ? p : -1;
    s_bits[i] = i / 64 == w ? 1ull << (i % 64) : 0ull;
    s_depth[i] = p >= 0;
  }
  if (bad && w == 0) record_error(9 /* FP8Q_ERR_RANGE */);
  if (__syncthreads_or(falls)) return;
  for (;;) {
    uint64_t add[ITEMS];
    int next[ITEMS], up[ITEMS];
    bool more = false;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
      const int i = tid + k * T, p = i < n ? s_anc[i] : -1;
      add[k] = p >= 0 ? s_bits[p] : 0ull;
      up[k] = p >= 0 ? s_depth[p] : 0;
      next[k] = p >= 0 ? s_anc[p] : -1;
      more |= next[k] >= 0;
    }
    more = __syncthreads_or(more);
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
      const int i = tid + k * T;
      if (i >= n) continue;
      s_bits[i] |= add[k];
      s_depth[i] += up[k];
      s_anc[i] = next[k];
    }
    __syncthreads();
    if (!more) break;
  }
  const int64_t c = a.positions && a.ctx_lens ? a.ctx_lens[b] : 0;
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    const int i = tid + k * T;
    if (i >= n) continue;
    a.mask[(first + i) * a.ldm + w] = static_cast<int64_t>(s_bits[i]);
    if (a.positions && w == 0) a.positions[first + i] = c + s_depth[i];
  }
}

// ---------------------------------------------------------------------------------------------
// Accepted rows to consecutive positions
// ---------------------------------------------------------------------------------------------
constexpr int kAcceptThreads = 128;
constexpr int kAcceptBatch = 8;      // rows in flight per thread

struct AcceptArgs {
  uint8_t *k_cache, *v_cache;        // [layers][num_slots][row], layer_stride bytes apart
  int64_t layer_stride, num_blocks;
  const int32_t *block_table;        // [B][max_blocks]
  int64_t max_blocks;
  uint32_t block_size;
  const int32_t *ctx_lens, *cu;      // [B], [B + 1]
  const int32_t *path;               // [B][max_path]
  int64_t max_path;
  const int32_t *path_lens;          // [B]
  int chunks;                        // 16-byte chunks per row
  int32_t *new_lens;                 // [B]
};

// One CTA per (sequence, layer).  The row of position ctx + path[k] goes to position ctx + k, k
// ascending.  path is strictly ascending, so path[k] >= k: a row is only overwritten by a move
// whose index is not below its own, and a thread that keeps its 16-byte columns to itself, and
// loads a batch of rows before storing it, reads every row before it is overwritten.  36 layers of 64
// sequences with up to 8 moved rows of 1 KB (75 MB read and written) take 16 us with nothing in L2,
// 4.6 TB/s of the copy rate's 6.5, and 11 where it holds them; one layer 3 to 5 us, the latency of the
// launch and of three dependent loads.
__global__ void __launch_bounds__(kAcceptThreads) k_kv_accept(const AcceptArgs a) {
  extern __shared__ int64_t s_slot[];                          // [max_path] source, then target
  const int b = blockIdx.x, tid = threadIdx.x;
  const int64_t layer = blockIdx.y;
  int64_t *s_src = s_slot, *s_dst = s_slot + a.max_path;
  const int64_t c = a.ctx_lens[b], n = static_cast<int64_t>(a.cu[b + 1]) - a.cu[b];
  const int64_t len = a.path_lens[b];
  const int64_t capacity = a.max_blocks * a.block_size;
  bool bad = c < 0 || n < 0 || len < 0 || len > n || len > a.max_path || c + n > capacity;
  if (!bad) {
    const int32_t *path = a.path + b * a.max_path, *table = a.block_table + b * a.max_blocks;
    for (int64_t k = tid; k < len; k += kAcceptThreads) {
      const int64_t p = path[k], before = k > 0 ? path[k - 1] : -1;
      if (p <= before || p >= n) {
        bad = true;
        continue;
      }
      const uint32_t from = static_cast<uint32_t>(c + p), to = static_cast<uint32_t>(c + k);
      const int32_t bf = table[from / a.block_size], bt = table[to / a.block_size];
      bad |= bf < 0 || bf >= a.num_blocks || bt < 0 || bt >= a.num_blocks;
      s_src[k] = static_cast<int64_t>(bf) * a.block_size + from % a.block_size;
      s_dst[k] = p == k ? -1 : static_cast<int64_t>(bt) * a.block_size + to % a.block_size;
    }
  }
  bad = __syncthreads_or(bad);
  if (tid == 0 && layer == 0) {
    if (bad) record_error(9 /* FP8Q_ERR_RANGE */);
    a.new_lens[b] = static_cast<int32_t>(bad ? c : c + len);
  }
  if (bad) return;
  const int64_t row = static_cast<int64_t>(a.chunks) * 16;
  for (int col = tid; col < 2 * a.chunks; col += kAcceptThreads) {
    uint8_t *base = (col < a.chunks ? a.k_cache + col * 16 : a.v_cache + (col - a.chunks) * 16) +
                    layer * a.layer_stride;
    for (int64_t k0 = 0; k0 < len; k0 += kAcceptBatch) {
      uint4 v[kAcceptBatch];
#pragma unroll
      for (int j = 0; j < kAcceptBatch; ++j)
        if (k0 + j < len && s_dst[k0 + j] >= 0)
          v[j] = *reinterpret_cast<const uint4 *>(base + s_src[k0 + j] * row);
#pragma unroll
      for (int j = 0; j < kAcceptBatch; ++j)
        if (k0 + j < len && s_dst[k0 + j] >= 0)
          *reinterpret_cast<uint4 *>(base + s_dst[k0 + j] * row) = v[j];
    }
  }
}

}  // namespace fp8q
