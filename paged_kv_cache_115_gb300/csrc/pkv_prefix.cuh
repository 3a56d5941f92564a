// Decode attention over a prefix that the whole batch shares and each
// sequence's own tokens behind it.
#pragma once

#include "pkv_attention_common.cuh"

namespace pkv {

struct PrefixParams {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  __nv_bfloat16* out;
  const int32_t* prefix_table;
  const int32_t* block_tables;
  const int32_t* cu;            // null: one query row per sequence
  const int32_t* lens;
  long long num_blocks;
  int prefix_len, max_blocks_per_seq, S, T, max_len, H_q, H_kv, block_size;
  float scale_log2;
};

// One CTA of 4 warps per (query row, KV head): each warp takes every fourth
// key with an online softmax, the four states are merged in shared memory.
template <int D>
__global__ void __launch_bounds__(128) prefix_simple_kernel(const __grid_constant__ PrefixParams p) {
  constexpr int E = D / 32;
  __shared__ float s_m[4][8], s_l[4][8], s_o[4][8][D];
  const int t = blockIdx.x, j = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait_primary();
  pdl_launch_dependents();
  const int K = p.block_size, G = p.H_q / p.H_kv;
  int s = t, i = 0, n = 1;
  if (p.cu != nullptr) {
    if (t >= p.cu[p.S]) return;
    int lo = 0, hi = p.S;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.cu[mid] <= t) lo = mid; else hi = mid;
    }
    s = lo;
    n = p.cu[s + 1] - p.cu[s];
    i = t - p.cu[s];
  }
  const int L = effective_len(p.lens[s], p.max_len, p.max_blocks_per_seq * K);
  if (p.cu != nullptr && n > L) {
    record_error(PKV_DEVERR_CONTEXT_LEN);
    return;
  }
  const int lim = L - n + i;                    // last visible key
  float q[8][E], o[8][E], m[8], l[8];
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    m[g] = -INFINITY;
    l[g] = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      o[g][e] = 0.f;
      q[g][e] = g < G ? __bfloat162float(p.q[((int64_t)t * p.H_q + j * G + g) * D + lane * E + e]) : 0.f;
    }
  }
  for (int x = warp; x <= lim; x += 4) {
    const int lb = x / K;
    const int32_t id = x < p.prefix_len ? p.prefix_table[lb]
                                        : p.block_tables[(int64_t)s * p.max_blocks_per_seq + lb];
    const bool good = id >= 0 && id < p.num_blocks;
    if (!good && lane == 0) record_error(PKV_DEVERR_BLOCK_ID);
    const int64_t at = (((int64_t)(good ? id : 0) * K + x % K) * p.H_kv + j) * D + lane * E;
    float kv[E], vv[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      kv[e] = good ? __bfloat162float(p.k[at + e]) : 0.f;
      vv[e] = good ? __bfloat162float(p.v[at + e]) : 0.f;
    }
    for (int g = 0; g < G; ++g) {
      float d = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) d += q[g][e] * kv[e];
      d = warp_sum(d) * p.scale_log2;
      const float mn = fmaxf(m[g], d), al = exp2f(m[g] - mn), w = exp2f(d - mn);
      m[g] = mn;
      l[g] = l[g] * al + w;
#pragma unroll
      for (int e = 0; e < E; ++e) o[g][e] = o[g][e] * al + w * vv[e];
    }
  }
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    if (lane == 0) {
      s_m[warp][g] = m[g];
      s_l[warp][g] = l[g];
    }
#pragma unroll
    for (int e = 0; e < E; ++e) s_o[warp][g][lane * E + e] = o[g][e];
  }
  __syncthreads();
  for (int x = threadIdx.x; x < G * D; x += 128) {
    const int g = x / D, d = x - g * D;
    float M = fmaxf(fmaxf(s_m[0][g], s_m[1][g]), fmaxf(s_m[2][g], s_m[3][g]));
    if (M == -INFINITY) M = 0.f;
    float lt = 0.f, ot = 0.f;
    for (int w = 0; w < 4; ++w) {
      const float f = exp2f(s_m[w][g] - M);
      lt += s_l[w][g] * f;
      ot += s_o[w][g][d] * f;
    }
    p.out[((int64_t)t * p.H_q + j * G + g) * D + d] = __float2bfloat16_rn(lt > 0.f ? ot / lt : 0.f);
  }
}

}  // namespace pkv
