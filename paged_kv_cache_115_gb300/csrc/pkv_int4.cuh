// 4-bit KV pages: quantizing writes and the description of a pool.
//
// Per token and KV head a row x of D values is stored as 4-bit codes with one
// bf16 scale s and one bf16 offset z:
//   z = min x rounded down to bf16, s = bf16((max x - z) / 15), r = 1 / s,
//   code = clamp(rint((x - z) r), 0, 15), read back as z + s code,
// all in float32 (each step rounded to nearest even), so that codes, scales and
// offsets are fixed to the bit.  Rounding z down keeps every x - z >= 0 whatever
// the row's distance from zero is next to its spread: the error stays below
// 0.57 s (half a step, and 15 codes of a scale that is off by 2^-8 at most).  A
// scale below 2^-126 has no float32 reciprocal: r = 0, the row reads as z (less
// than 2^-122 off).  A row
// with a NaN or an infinity (or whose offset or scale overflows) gets s = z = NaN
// and reads as NaN, as it would in a bf16 pool.
//
// Element 2 i of a row is the low half of its byte i.  A token's (s, z) is one
// 32-bit word, s in the low half; the words of a pool are [num_blocks, H_kv,
// block_size], so that the words of a block's tokens lie together for each head.
#pragma once

#include "pkv_device.cuh"

namespace pkv {

__device__ __forceinline__ float int4_scale(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float int4_offset(uint32_t w) {
  return __uint_as_float(w & 0xffff0000u);
}

struct Int4Row {
  float z, r;
  uint32_t word;     // (s, z) as stored
  bool bad;          // not finite: codes 0
};

// From a row's least and largest value and whether all of it is finite.
__device__ __forceinline__ Int4Row int4_row(float lo, float hi, bool finite) {
  Int4Row q;
  const __nv_bfloat16 z = __float2bfloat16_rd(lo);
  q.z = __bfloat162float(z);
  const __nv_bfloat16 s = __float2bfloat16_rn(__fdiv_rn(hi - q.z, 15.f));
  const float sf = __bfloat162float(s);
  q.bad = !finite || !(fabsf(q.z) < INFINITY) || !(sf < INFINITY);
  q.r = sf >= 1.17549435e-38f ? __frcp_rn(sf) : 0.f;
  q.word = q.bad ? 0x7fff7fffu
                 : (uint32_t)__bfloat16_as_ushort(s) | (uint32_t)__bfloat16_as_ushort(z) << 16;
  return q;
}

// N codes (4 or 8) packed, the first in the lowest bits.  (x - z) r of a finite row
// lies in [0, 15.1): the clamp of the definition changes nothing.  Adding 1.5 * 2^23
// rounds to nearest even into the low bits, and the constant's own bits come off
// the packed word at once.
template <int N>
__device__ __forceinline__ uint32_t int4_pack(const Int4Row& q, const float* x) {
  constexpr uint32_t kMagic = 0x4b400000u;      // 12582912.0f
  uint32_t w = 0, off = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    w += __float_as_uint(__fmul_rn(x[i] - q.z, q.r) + 12582912.f) << (4 * i);
    off += kMagic << (4 * i);
  }
  w -= off;
  if constexpr (N < 8) w &= (1u << (4 * N)) - 1;
  return q.bad ? 0u : w;
}

// Least and largest value, NaN once there is one.
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

struct Int4WriteParams {
  const void* k;
  const void* v;
  int64_t k_stride, v_stride;        // elements between tokens
  const int64_t* slots;              // or null: slots from positions and tables
  const int32_t* positions;
  const int32_t* block_tables;       // row i of token i
  int64_t* slots_out;                // may be null (with tables)
  uint8_t* k_cache;
  uint8_t* v_cache;
  uint32_t* k_words;
  uint32_t* v_words;
  int64_t num_blocks;
  int max_blocks, block_size, log2_bs;
  int T, H;
};

constexpr int kInt4Threads = 256;
constexpr int kInt4Loads = 4;            // 16-byte loads a lane

// A row takes LANES lanes of four 16-byte blocks each (32 bf16 or 16 float32 values):
// what is done once a row (scale, reciprocal, slot) counts for many values, and a
// lane has 64 bytes in flight.  WIDE: rows on 16-byte boundaries, else value by value.
// Bound by HBM: (2 e D + D + 8) H bytes a token.  16381 tokens of 8 heads of 128 in
// bf16: 17.8 us, 4.8 TB/s with the call (a lane to 16 bytes, which repeats the row's
// work eight times: 47 us); 64 tokens: 9.5 us, the host's.
template <typename TIN, int D, bool WIDE>
__global__ void __launch_bounds__(kInt4Threads)
kv_write_int4_kernel(const __grid_constant__ Int4WriteParams p) {
  constexpr int V = 16 / sizeof(TIN), LANES = D / (V * kInt4Loads), RPI = kInt4Threads / LANES;
  pdl_wait_primary();
  pdl_launch_dependents();
  const int li = threadIdx.x % LANES;
  const unsigned rows = 2 * p.H;                 // of a token: K heads, V heads
  const unsigned r = blockIdx.x * RPI + threadIdx.x / LANES;
  const bool in = r < (unsigned)p.T * rows;      // below 2^31
  const int t = in ? (int)(r / rows) : 0;
  const int zh = (int)(r - (unsigned)t * rows);
  const bool z = zh >= p.H;
  const int h = zh - (z ? p.H : 0);
  const TIN* src = static_cast<const TIN*>(z ? p.v : p.k) + t * (z ? p.v_stride : p.k_stride) +
                   (in ? h * D : 0);
  // (the rows are read before their slots are known: one wait for memory, not two)
  uint4 raw[kInt4Loads];
  if constexpr (WIDE) {
#pragma unroll
    for (int i = 0; i < kInt4Loads; ++i)
      raw[i] = in ? __ldcs(reinterpret_cast<const uint4*>(src) + i * LANES + li) : make_uint4(0, 0, 0, 0);
  }
  int64_t blk = -1;
  int off = 0;
  if (in) {
    const bool leader = zh == 0 && li == 0;
    if (p.slots != nullptr) {
      const int64_t slot = p.slots[t];
      const int64_t b = p.log2_bs >= 0 ? slot >> p.log2_bs : slot / p.block_size;
      if (slot >= 0 && b < p.num_blocks) {
        blk = b;
        off = (int)(slot - b * p.block_size);
      } else if (slot != -1 && leader) {
        record_error(PKV_DEVERR_SLOT);
      }
    } else {
      const int pos = p.positions[t];
      if (pos >= 0) {
        const int lb = p.log2_bs >= 0 ? pos >> p.log2_bs : pos / p.block_size;
        if (lb >= p.max_blocks) {
          if (leader) record_error(PKV_DEVERR_POSITION);
        } else {
          const int64_t phys = p.block_tables[(int64_t)t * p.max_blocks + lb];
          if (phys < 0 || phys >= p.num_blocks) {
            if (leader) record_error(PKV_DEVERR_BLOCK_ID);
          } else {
            blk = phys;
            off = pos - lb * p.block_size;
          }
        }
      }
      if (leader && p.slots_out != nullptr) p.slots_out[t] = blk < 0 ? -1 : blk * p.block_size + off;
    }
  }
  float x[kInt4Loads][V];
#pragma unroll
  for (int i = 0; i < kInt4Loads; ++i) {
    if constexpr (!WIDE) {
#pragma unroll
      for (int e = 0; e < V; ++e) x[i][e] = in ? to_f32(src[(i * LANES + li) * V + e]) : 0.f;
    } else {
      const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (sizeof(TIN) == 4) {
          x[i][e] = __uint_as_float(w[e]);
        } else {
          x[i][2 * e] = __uint_as_float(w[e] << 16);
          x[i][2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
        }
      }
    }
  }
  float lo = x[0][0], hi = x[0][0];
#pragma unroll
  for (int i = 0; i < kInt4Loads; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) {
      lo = min_nan(lo, x[i][e]);
      hi = max_nan(hi, x[i][e]);
    }
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) {
    lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  if (blk < 0) return;
  const Int4Row q = int4_row(lo, hi, fabsf(lo) < INFINITY && fabsf(hi) < INFINITY);
  uint8_t* dst = (z ? p.v_cache : p.k_cache) + ((blk * p.block_size + off) * p.H + h) * (D / 2);
#pragma unroll
  for (int i = 0; i < kInt4Loads; ++i) {
    uint8_t* d = dst + (i * LANES + li) * (V / 2);
    if constexpr (V == 8) *reinterpret_cast<uint32_t*>(d) = int4_pack<8>(q, x[i]);
    else *reinterpret_cast<uint16_t*>(d) = (uint16_t)int4_pack<4>(q, x[i]);
  }
  if (li == 0) (z ? p.v_words : p.k_words)[(blk * p.H + h) * p.block_size + off] = q.word;
}

}  // namespace pkv
