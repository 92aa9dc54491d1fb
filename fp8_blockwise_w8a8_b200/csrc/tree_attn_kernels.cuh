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
#include <cuda_fp8.h>
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
  float *ws;
  uint16_t *out;               // [total][ldo] bf16
  int64_t ldo;
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

// One warp per (node, head): lanes share the dims, positions in order.
template <int D>
__global__ void __launch_bounds__(128) k_tree_attn(const TreeAttnArgs a) {
  constexpr int N = D / 32;
  const int b = blockIdx.z, h = blockIdx.y, lane = threadIdx.x & 31;
  const int i = blockIdx.x * 4 + (threadIdx.x >> 5);
  const TreeSeq s = tree_seq(a, b, blockIdx.x == 0 && h == 0 && threadIdx.x == 0);
  if (i >= s.n) return;
  const int g = h / (a.Hq / a.Hkv);
  const float c2 = a.sm_scale * a.scale3[0] * a.scale3[1] * 1.4426950408889634f;
  const int64_t row = static_cast<int64_t>(a.Hkv) * D;
  float q[N], o[N], m = -INFINITY, l = 0.0f;
  auto dec = [](uint8_t c) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
  };
  for (int d = 0; d < N; ++d) {
    q[d] = dec(a.q[(s.first + i) * a.ldq + h * D + lane * N + d]);
    o[d] = 0.0f;
  }
  for (int j = 0; j < s.ctx + i + 1; ++j) {
    const int nj = j - s.ctx;
    if (nj >= 0 && a.mask && !((a.mask[(s.first + i) * a.ldm + nj / 64] >> (nj % 64)) & 1)) continue;
    const int32_t blk = a.block_table[b * a.max_blocks + j / a.block_size];
    if (blk < 0 || blk >= a.num_blocks) {
      record_error(9 /* FP8Q_ERR_RANGE */);
      continue;
    }
    const int64_t at = (static_cast<int64_t>(blk) * a.block_size + j % a.block_size) * row + g * D +
                       lane * N;
    float z = 0.0f;
    for (int d = 0; d < N; ++d) z = fmaf(q[d], dec(a.k_cache[at + d]), z);
#pragma unroll
    for (int x = 16; x; x >>= 1) z += __shfl_xor_sync(0xffffffffu, z, x);
    z *= c2;
    const float m2 = fmaxf(m, z), f = m2 == m ? 1.0f : exp2f(m - m2), p = exp2f(z - m2);
    m = m2;
    l = fmaf(l, f, p);
    for (int d = 0; d < N; ++d) o[d] = fmaf(o[d], f, p * dec(a.v_cache[at + d]));
  }
  for (int d = 0; d < N; ++d) {
    const __nv_bfloat16 r = __float2bfloat16_rn(l == 0.0f ? 0.0f : a.scale3[2] * (o[d] / l));
    a.out[(s.first + i) * a.ldo + h * D + lane * N + d] = *reinterpret_cast<const uint16_t *>(&r);
  }
}

}  // namespace fp8q
