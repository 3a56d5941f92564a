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

// INT8 pools: the token's K and V rows stand in s_all; each gets its scale
// max|x| / 127 and codes rint(x / scale), as kv_append_quant_kernel makes them.
// Called by the whole CTA of W warps.
template <int W>
__device__ __forceinline__ void rope_int8_rows(const RopeParams& p, int64_t slot,
                                               int64_t pool_row, const float (&amax)[2],
                                               const float* s_all, float (*s_amax)[W]) {
  if (slot < 0) return;
  const int n = p.H_kv * p.D;
#pragma unroll
  for (int z = 0; z < 2; ++z) {
    const float m = warp_max(amax[z]);
    if ((threadIdx.x & 31) == 0) s_amax[z][threadIdx.x >> 5] = m;
  }
  __syncthreads();
#pragma unroll
  for (int z = 0; z < 2; ++z) {
    float m = s_amax[z][0];
#pragma unroll
    for (int i = 1; i < W; ++i) m = fmaxf(m, s_amax[z][i]);
    const float sc = m == 0.f ? 0.f : __fdiv_rn(m, 127.f);
    int8_t* dst = reinterpret_cast<int8_t*>(z ? p.v_cache : p.k_cache) + pool_row;
    for (int e = threadIdx.x; e < n; e += W * 32) {
      const float c = sc == 0.f ? 0.f : rintf(__fdiv_rn(s_all[z * n + e], sc));
      dst[e] = (int8_t)fminf(127.f, fmaxf(-127.f, c));
    }
    if (threadIdx.x == 0) (z ? p.v_ts : p.k_ts)[slot] = sc;
  }
}

// Any even head_dim up to 512: one CTA per token, one warp per head row, the
// row in shared memory (a rotated pair may sit in two lanes).
template <typename TIN, int FMT>
__global__ void __launch_bounds__(kRopeThreads)
rope_any_kernel(const __grid_constant__ RopeParams p) {
  constexpr int W = kRopeThreads / 32;
  __shared__ float s_row[W][kRopeMaxDim];
  __shared__ float s_amax[2][W];
  extern __shared__ float s_all[];            // INT8: the token's K, then V row
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
  const float amax[2] = {amax_k, amax_v};
  if constexpr (FMT == 2) rope_int8_rows<W>(p, slot, pool_row, amax, s_all, s_amax);
}

// Vectorised form: head_dim 64 or 128 (256 for bf16), rows and strides on
// 16-byte boundaries, the rotation in whole lanes.  A lane holds V = 16 /
// sizeof(TIN) values of a row, so a row takes D / V lanes and a CTA 256 V / D
// rows at once (16 for bf16 at head_dim 128).  One CTA per token: its rows
// (query heads, key heads, value heads) are loaded four to a thread before
// any is used, the cosines and sines of a lane once per token.  A rotated
// pair sits in one lane (interleaved) or in two lanes half a rotation apart
// (a shuffle per value).
// Bound by HBM: 2 (H_q + H_kv) D e + (2 H_kv D) e bytes a token.
template <typename TIN>
__device__ __forceinline__ void rope_unpack(const uint4& r, float (&x)[16 / sizeof(TIN)]) {
  if constexpr (sizeof(TIN) == 4) {
    x[0] = __uint_as_float(r.x); x[1] = __uint_as_float(r.y);
    x[2] = __uint_as_float(r.z); x[3] = __uint_as_float(r.w);
  } else {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

template <typename TIN>
__device__ __forceinline__ uint4 rope_pack(const float (&x)[16 / sizeof(TIN)]) {
  if constexpr (sizeof(TIN) == 4)
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3]));
  else
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
}

// V values as e4m3 codes of x / scale, V bytes.
template <int V>
__device__ __forceinline__ void rope_store_fp8(uint8_t* dst, const float (&x)[V], float scale) {
  uint32_t w[V / 4];
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(
        make_float2(__fdiv_rn(x[4 * i], scale), __fdiv_rn(x[4 * i + 1], scale)), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(
        make_float2(__fdiv_rn(x[4 * i + 2], scale), __fdiv_rn(x[4 * i + 3], scale)), __NV_SATFINITE, __NV_E4M3);
    w[i] = lo | (hi << 16);
  }
  if constexpr (V == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  else *reinterpret_cast<uint32_t*>(dst) = w[0];
}

template <typename TIN, int FMT, int D, bool PAIRS>
__global__ void __launch_bounds__(kRopeThreads)
rope_vec_kernel(const __grid_constant__ RopeParams p) {
  constexpr int V = 16 / sizeof(TIN), LANES = D / V, RPI = kRopeThreads / LANES, BATCH = 4;
  static_assert(LANES <= 32, "a row must fit a warp");
  constexpr int W = kRopeThreads / 32;
  __shared__ float s_amax[2][W];
  extern __shared__ float s_all[];              // INT8: the token's K, then V row
  const int tid = threadIdx.x, lane = tid & 31;
  const int e0 = (tid % LANES) * V, rg = tid / LANES;
  const int t = blockIdx.x;
  pdl_wait_primary();
  pdl_launch_dependents();
  const int pos = p.positions[t];
  int64_t slot = p.slots[t];
  const int HK = p.H_q + p.H_kv, rows = HK + p.H_kv;
  const TIN* q = static_cast<const TIN*>(p.q) + t * p.q_stride;
  const TIN* k = static_cast<const TIN*>(p.k) + t * p.k_stride;
  const TIN* v = static_cast<const TIN*>(p.v) + t * p.v_stride;
  TIN* qo = static_cast<TIN*>(p.q_out) + t * p.qo_stride;
  auto source = [&](int r) -> const TIN* {
    return (r < p.H_q ? q + r * D : (r < HK ? k + (r - p.H_q) * D : v + (r - HK) * D)) + e0;
  };
  if (pos < 0) return;                          // padding
  if (pos >= p.max_pos) {
    if (tid == 0) record_error(PKV_DEVERR_POSITION);
    return;
  }
  if (slot < 0 || slot >= p.num_slots) {
    if (slot != -1 && tid == 0) record_error(PKV_DEVERR_SLOT);
    slot = -1;
  }
  uint4 raw[BATCH];
#pragma unroll
  for (int b = 0; b < BATCH; ++b)
    if (b * RPI + rg < rows) raw[b] = __ldcs(reinterpret_cast<const uint4*>(source(b * RPI + rg)));
  // cosines and sines of this lane's values (1, 0 behind the rotation)
  const int half = p.rot >> 1;
  constexpr int NC = PAIRS ? V / 2 : V;
  float c[NC], s[NC];
  const bool turned = e0 < p.rot, second = !PAIRS && e0 >= half;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    c[i] = 1.f;
    s[i] = 0.f;
  }
  if (turned) {
    const float* cs = p.cos_sin + (int64_t)pos * p.rot + (PAIRS ? e0 >> 1 : (second ? e0 - half : e0));
#pragma unroll
    for (int i = 0; i < NC; i += 2) {
      const float2 a = __ldg(reinterpret_cast<const float2*>(cs + i));
      const float2 b = __ldg(reinterpret_cast<const float2*>(cs + half + i));
      c[i] = a.x; c[i + 1] = a.y;
      s[i] = b.x; s[i + 1] = b.y;
    }
    if (!PAIRS && !second) {                    // the first of a pair takes off
#pragma unroll
      for (int i = 0; i < NC; ++i) s[i] = -s[i];
    }
  }
  // lane that holds the other value of this lane's pairs
  const int mate = PAIRS || !turned ? lane : (second ? lane - half / V : lane + half / V);
  uint4 wq = make_uint4(0, 0, 0, 0), wk = wq;
  if (p.wq != nullptr) wq = __ldg(reinterpret_cast<const uint4*>(static_cast<const TIN*>(p.wq) + e0));
  if (p.wk != nullptr) wk = __ldg(reinterpret_cast<const uint4*>(static_cast<const TIN*>(p.wk) + e0));
  const int64_t pool_row = slot * p.H_kv * D;
  float amax[2] = {0.f, 0.f};

  for (int r0 = 0; r0 < rows; r0 += RPI * BATCH) {
    if (r0 > 0) {
#pragma unroll
      for (int b = 0; b < BATCH; ++b)
        if (r0 + b * RPI + rg < rows)
          raw[b] = __ldcs(reinterpret_cast<const uint4*>(source(r0 + b * RPI + rg)));
    }
#pragma unroll
    for (int b = 0; b < BATCH; ++b) {
      if (r0 + b * RPI >= rows) break;          // the same for the whole CTA: shuffles stay whole
      const int r = r0 + b * RPI + rg;
      const int z = r < p.H_q ? 0 : (r < HK ? 1 : 2);               // q, k, v (or past the end)
      float x[V];
      rope_unpack<TIN>(raw[b], x);
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (z < 2 && (z ? p.wk : p.wq) != nullptr) {
        float w[V];
        rope_unpack<TIN>(z ? wk : wq, w);
        const float inv = rsqrtf(ss / D + p.eps);
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] *= inv * w[i];
      }
      float y[V];
      if constexpr (PAIRS) {
#pragma unroll
        for (int i = 0; i < V; i += 2) {
          y[i] = x[i] * c[i / 2] - x[i + 1] * s[i / 2];
          y[i + 1] = x[i + 1] * c[i / 2] + x[i] * s[i / 2];
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float o = __shfl_sync(0xffffffffu, x[i], mate);
          y[i] = x[i] * c[i] + o * s[i];
        }
      }
      if (r >= rows) continue;
      if (z == 0) {
        *reinterpret_cast<uint4*>(qo + r * D + e0) = rope_pack<TIN>(y);
        continue;
      }
      if (slot < 0) continue;
      const int at = (z == 1 ? r - p.H_q : r - HK) * D + e0;        // in the token's K or V row
      if constexpr (FMT == 2) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float val = z == 1 ? y[i] : x[i];
          s_all[(z - 1) * p.H_kv * D + at + i] = val;
          amax[z - 1] = fmaxf(amax[z - 1], fabsf(val));
        }
      } else if (z == 1) {
        if constexpr (FMT == 0) {
          reinterpret_cast<uint4*>(p.k_cache)[(pool_row + at) / V] = rope_pack<TIN>(y);
        } else if constexpr (FMT == 3) {
          uint32_t* dst = reinterpret_cast<uint32_t*>(p.k_cache + 2 * (pool_row + at));
#pragma unroll
          for (int i = 0; i < V / 2; ++i) dst[i] = pack_bf16x2(y[2 * i], y[2 * i + 1]);
        } else {
          rope_store_fp8<V>(p.k_cache + pool_row + at, y, p.k_scale);
        }
      } else {
        if constexpr (FMT == 0) reinterpret_cast<uint4*>(p.v_cache)[(pool_row + at) / V] = raw[b];
        else rope_store_fp8<V>(p.v_cache + pool_row + at, x, p.v_scale);
      }
    }
  }
  if constexpr (FMT == 2) rope_int8_rows<W>(p, slot, pool_row, amax, s_all, s_amax);
}

}  // namespace pkv
