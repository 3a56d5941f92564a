// Head norms, rotation by position and KV append of new tokens in one pass.
//
// For a query or key head row x: y = x rsqrt(mean(x^2) + eps) w, then each
// pair (a, b) of rotated values becomes (a c - b s, b c + a s) with the
// position's cosine and sine from a float32 table.  Query rows go to q_out,
// key rows (and V rows as they are) to the token's slot of the pools.
// Everything between the load and the store is float32; a value is rounded
// once, to the type it is stored in.
#pragma once

#include "pkv_copy.cuh"

namespace pkv {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxDim = 512;
constexpr int kRopeMaxInt8Row = 8192;   // floats of one token's K or V row in shared memory

struct RopeParams {
  const void* q;
  const void* k;
  const void* v;
  const void* wq;              // null: no norm
  const void* wk;
  const int32_t* positions;
  const float* cos_sin;
  const int64_t* slots;
  void* q_out;
  uint8_t* k_cache;
  uint8_t* v_cache;
  float* k_ts;                 // INT8 pools: scale per slot
  float* v_ts;
  int64_t q_stride, k_stride, v_stride, qo_stride;   // elements between tokens
  int64_t num_slots;
  float eps, k_scale, v_scale;
  int T, H_q, H_kv, D, rot, max_pos, interleaved;
};

// Stores value x of element e of a K (z 0) or V (z 1) row at `base` elements
// into the pool; FMT as in kv_append_quant_kernel, 0 plain.
template <typename TIN, int FMT>
__device__ __forceinline__ void rope_store(const RopeParams& p, int z, int64_t at, float x) {
  uint8_t* pool = z ? p.v_cache : p.k_cache;
  if constexpr (FMT == 0) {
    reinterpret_cast<TIN*>(pool)[at] = from_f32<TIN>(x);
  } else if constexpr (FMT == 3) {
    if (z == 0) reinterpret_cast<__nv_bfloat16*>(pool)[at] = __float2bfloat16_rn(x);
    else pool[at] = f32_to_e4m3(__fdiv_rn(x, p.v_scale));
  } else {
    pool[at] = f32_to_e4m3(__fdiv_rn(x, z ? p.v_scale : p.k_scale));
  }
}

// Any even head_dim up to 512: one CTA per token, one warp per head row, the
// row in shared memory (a rotated pair may sit in two lanes).
template <typename TIN, int FMT>
__global__ void __launch_bounds__(kRopeThreads)
rope_any_kernel(const __grid_constant__ RopeParams p) {
  constexpr int W = kRopeThreads / 32;
  __shared__ float s_row[W][kRopeMaxDim];
  __shared__ float s_amax[W];
  extern __shared__ float s_all[];            // INT8: the token's K (then V) row
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x;
  pdl_wait_primary();
  pdl_launch_dependents();
  const int pos = p.positions[t];
  if (pos < 0) return;                        // padding
  if (pos >= p.max_pos) {
    if (threadIdx.x == 0) record_error(PKV_DEVERR_POSITION);
    return;
  }
  int64_t slot = p.slots[t];
  if (slot < 0 || slot >= p.num_slots) {
    if (slot != -1 && threadIdx.x == 0) record_error(PKV_DEVERR_SLOT);
    slot = -1;
  }
  const int D = p.D, half = p.rot / 2;
  const float* cs = p.cos_sin + (int64_t)pos * p.rot;
  const int rows = p.H_q + 2 * p.H_kv;
  const int64_t pool_row = slot * p.H_kv * D;
  float amax_k = 0.f, amax_v = 0.f;
  for (int r = warp; r < rows; r += W) {
    const int z = r < p.H_q ? 0 : (r < p.H_q + p.H_kv ? 1 : 2);      // q, k, v
    const int h = z == 0 ? r : r - p.H_q - (z == 2 ? p.H_kv : 0);
    if (z && slot < 0) continue;
    const TIN* src = static_cast<const TIN*>(z == 0 ? p.q : (z == 1 ? p.k : p.v)) +
                     t * (z == 0 ? p.q_stride : (z == 1 ? p.k_stride : p.v_stride)) + h * D;
    const TIN* w = static_cast<const TIN*>(z == 0 ? p.wq : (z == 1 ? p.wk : nullptr));
    float ss = 0.f;
    for (int e = lane; e < D; e += 32) {
      const float x = to_f32(src[e]);
      s_row[warp][e] = x;
      ss += x * x;
    }
    if (z < 2 && w != nullptr) {
      const float inv = rsqrtf(warp_sum(ss) / D + p.eps);
      for (int e = lane; e < D; e += 32) s_row[warp][e] *= inv * to_f32(w[e]);
    }
    __syncwarp();
    for (int e = lane; e < D; e += 32) {
      float y = s_row[warp][e];
      if (z < 2 && e < p.rot) {
        const int i = p.interleaved ? e >> 1 : (e < half ? e : e - half);
        const bool second = p.interleaved ? (e & 1) : e >= half;
        const float o = s_row[warp][p.interleaved ? e ^ 1 : (second ? e - half : e + half)];
        const float c = cs[i], s = cs[half + i];
        y = second ? y * c + o * s : y * c - o * s;
      }
      if (z == 0) {
        static_cast<TIN*>(p.q_out)[t * p.qo_stride + h * D + e] = from_f32<TIN>(y);
      } else if constexpr (FMT == 2) {
        s_all[(z - 1) * p.H_kv * D + h * D + e] = y;
        if (z == 1) amax_k = fmaxf(amax_k, fabsf(y)); else amax_v = fmaxf(amax_v, fabsf(y));
      } else {
        rope_store<TIN, FMT>(p, z - 1, pool_row + h * D + e, y);
      }
    }
    __syncwarp();
  }
  if constexpr (FMT == 2) {
    if (slot < 0) return;
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const float m = warp_max(z ? amax_v : amax_k);
      __syncthreads();
      if (lane == 0) s_amax[warp] = m;
      __syncthreads();
      float amax = s_amax[0];
#pragma unroll
      for (int i = 1; i < W; ++i) amax = fmaxf(amax, s_amax[i]);
      const float sc = amax == 0.f ? 0.f : __fdiv_rn(amax, 127.f);
      int8_t* dst = reinterpret_cast<int8_t*>(z ? p.v_cache : p.k_cache) + pool_row;
      for (int e = threadIdx.x; e < p.H_kv * D; e += kRopeThreads) {
        float c = sc == 0.f ? 0.f : rintf(__fdiv_rn(s_all[z * p.H_kv * D + e], sc));
        dst[e] = (int8_t)fminf(127.f, fmaxf(-127.f, c));
      }
      if (threadIdx.x == 0) (z ? p.v_ts : p.k_ts)[slot] = sc;
    }
  }
}

}  // namespace pkv
