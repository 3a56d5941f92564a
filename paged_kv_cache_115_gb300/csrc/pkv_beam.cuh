// Selection of beam search: the best candidates over a request's beams and the
// vocabulary, from the model's output and the beams' scores.
//
//   candidate (b, v) = score_b + logit_bv - log sum_v' exp(logit_bv'),
// ordered by value, then by the lowest b V + v.  One pass over the logits: a CTA
// takes a tile of a row into registers and leaves the tile's largest logit m,
// its sum of exp(x - m) and its best candidates; a second kernel joins the tiles
// of a request's beams.  A row's order among its own candidates is that of its
// logits, so the sum is only needed there; joined in 64 bits, because candidates
// of two beams may lie next to each other.
#pragma once

#include "pkv_device.cuh"

namespace pkv {

constexpr int kBeamThreads = 256;
constexpr int kBeamWarps = kBeamThreads / 32;
constexpr int kBeamMax = 32;                 // beams of a request, candidates asked for
constexpr int kBeamBuffer = 512;             // candidates at or above a tile's bound

struct BeamParams {
  const void* logits;
  int64_t stride;              // elements between rows
  const float* scores;         // [R][B]
  const uint8_t* finished;     // [R][B] or null
  int32_t* tokens;             // [R][N]
  int32_t* parents;
  float* scores_out;
  uint8_t* finished_out;       // or null
  float2* tile_ms;             // [R B][tiles]: m, sum of exp(x - m)
  float* tile_x;               // [R B][tiles][N]: best logits of a tile, -inf: none
  int32_t* tile_v;             // and their tokens
  int R, B, V, N, tiles, eos;
};

// A bound of the warp: at least n of its lanes' values are at or above it (0 with
// fewer than n lanes that have one).  The n-th largest but for equal values, which
// count once.
__device__ __forceinline__ uint32_t warp_bound(uint32_t x, int n) {
  uint32_t top = 0;
  for (int i = 0; i < n; ++i) {
    top = __reduce_max_sync(0xffffffffu, x);
    if (x == top) x = 0;
  }
  return top;
}

// The sum of exp(x) is kept as s 2^b, b = beam_base(m) whole: terms 2^(x c - b) with c
// the float32 next to log2 e, one fused operation an argument, and sums of different
// tiles join by exact powers of two.  Far from zero (a row of masks at the type's
// lowest value) whole b no longer serve: there s is the sum of exp(x - m).
constexpr float kBeamLog2e = 1.44269504f;
__device__ __forceinline__ float beam_base(float m) { return ceilf(m * kBeamLog2e); }
// 2^d of a whole d <= 0
__device__ __forceinline__ float beam_pow2(float d) {
  return d < -126.f ? 0.f : __uint_as_float((uint32_t)((int)d + 127) << 23);
}

__device__ __forceinline__ bool beam_far(float m) { return !(fabsf(m) < 65536.f); }
// s of a part with maximum m as a share of a whole with maximum M >= m.  Where either
// is far, through the distance m - M and what either's base lies above its maximum (0
// to 1: one fused operation, since b and m c themselves are large there).
__device__ __forceinline__ float beam_join(float m, float s, float M) {
  if (m == -INFINITY) return s;                    // 0, or NaN
  const bool fm = beam_far(m), fM = beam_far(M);
  if (!fm && !fM) return s * beam_pow2(beam_base(m) - beam_base(M));
  const float up = fm ? 0.f : -fmaf(m, kBeamLog2e, -beam_base(m));
  const float down = fM ? 0.f : -fmaf(M, kBeamLog2e, -beam_base(M));
  return s * exp2f(fmaf(m - M, kBeamLog2e, up - down));
}

// A value's bits in its order (adding 0 makes one of the two zeros).
__device__ __forceinline__ uint32_t beam_order(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
// (by its bits alone: 64-bit floating-point operations are rare here; 0 for a value
// that is not finite)
__device__ __forceinline__ uint64_t beam_order(double x) {
  uint64_t b = (uint64_t)__double_as_longlong(x);
  if ((b << 1) == 0) b = 0;
  if ((b & 0x7ff0000000000000ull) == 0x7ff0000000000000ull) return 0;
  return b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull);
}

// The larger of each half of two bf16 pairs (a NaN gives way).
__device__ __forceinline__ uint32_t bf16x2_max(uint32_t a, uint32_t b) {
  const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                   *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&m);
}
// The largest value of a 16-byte block.
template <typename T>
__device__ __forceinline__ float beam_block_max(const uint4& r) {
  if constexpr (sizeof(T) == 4)
    return fmaxf(fmaxf(__uint_as_float(r.x), __uint_as_float(r.y)),
                 fmaxf(__uint_as_float(r.z), __uint_as_float(r.w)));
  const uint32_t m = bf16x2_max(bf16x2_max(r.x, r.y), bf16x2_max(r.z, r.w));
  return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
}

// Value e of a block, unpacked by an asm that is not shared between its uses: the
// compiler then keeps the block packed instead of all 64 values in registers.
template <typename T>
__device__ __forceinline__ float beam_value(const uint4& r, int e) {
  constexpr int P = sizeof(T) == 4 ? 1 : 2;
  const uint32_t w = e / P == 0 ? r.x : (e / P == 1 ? r.y : (e / P == 2 ? r.z : r.w));
  if constexpr (sizeof(T) == 4) return __uint_as_float(w);
  uint32_t x;
  if (e & 1) asm volatile("and.b32 %0, %1, 0xffff0000;" : "=r"(x) : "r"(w));
  else asm volatile("shl.b32 %0, %1, 16;" : "=r"(x) : "r"(w));
  return __uint_as_float(x);
}
__device__ __forceinline__ uint64_t beam_key(float x, int v) {
  return (uint64_t)beam_order(x) << 32 | (0xffffffffu - (uint32_t)v);
}

// A block's values at or above tau into the buffer (first value: token v).
template <typename T>
__device__ __noinline__ void beam_push(uint4 r, int v, uint32_t tau, int* n, uint64_t* key) {
#pragma unroll
  for (int e = 0; e < (int)(16 / sizeof(T)); ++e) {
    const float x = beam_value<T>(r, e);
    if (x > -INFINITY && beam_order(x) >= tau) {
      const int i = atomicAdd(n, 1);
      if (i < kBeamBuffer) key[i] = beam_key(x, v + e);
    }
  }
}

// Values lead .. of a block and the next one's behind them: the unaligned block of a
// row whose first value is value `lead` of an aligned one.
template <typename T>
__device__ __forceinline__ uint4 beam_shift(const uint4& lo, const uint4& hi, int lead) {
  const int bytes = lead * (int)sizeof(T);
  uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
  for (int i = 0; i < 6; ++i) w[i] = (bytes & 8) ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) w[i] = (bytes & 4) ? w[i + 1] : w[i];
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], (bytes & 2) * 8);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A tile of very many equal values: its N best one after the other, read again.
template <typename T, int NV>
__device__ __noinline__ void beam_tile_slow(const T* base, int V, int first, int N, float* out_x,
                                            int32_t* out_v, uint64_t* s_best) {
  constexpr int VE = 16 / sizeof(T);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int end = min(V, first + kBeamThreads * NV * VE);
  uint64_t last = ~0ull;
  for (int r = 0; r < N; ++r) {
    uint64_t best = 0;
    for (int v = first + threadIdx.x; v < end; v += kBeamThreads) {
      const float x = to_f32(base[v]);
      const uint64_t key = beam_key(x, v);
      if (x > -INFINITY && key < last && key > best) best = key;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const uint64_t y = __shfl_xor_sync(0xffffffffu, best, o);
      best = y > best ? y : best;
    }
    __syncthreads();
    if (lane == 0) s_best[warp] = best;
    __syncthreads();
    best = s_best[0];
#pragma unroll
    for (int w = 1; w < kBeamWarps; ++w) best = s_best[w] > best ? s_best[w] : best;
    last = best;
    if (threadIdx.x == 0) {                         // (more than kBeamBuffer values: there are N)
      const uint32_t o = (uint32_t)(best >> 32);
      out_x[r] = __uint_as_float(o ^ ((uint32_t)((int32_t)~o >> 31) | 0x80000000u));
      out_v[r] = (int32_t)(0xffffffffu - (uint32_t)best);
    }
  }
}

// NV 16-byte blocks a thread, all in flight at once: a tile of a row.  Rows of an odd
// vocabulary start anywhere: a block is then cut out of two aligned ones (the second
// comes from L1), so that a thread holds the same tokens, and a row's sum is the same
// to the last bit, wherever the row lies: rows alike tie.  What does not belong to the
// row counts as -inf.  Four CTAs an SM
// (three for float32): the blocks stay packed in registers and are unpacked as they are used.
// Bound by HBM (V e bytes a row) from afar: 512 rows of 131072 bf16 values in 38.5 us, of a
// whole call's 49 where a copy would take 19; what a warp issues for the bound (the N-th
// largest of the threads' maxima: with one over the warps' eight, 57 values a tile
// went through and the call took 85 us) and a CTA's chain of loads, exponents and
// reductions are the rest.  Equal values count once in the bound: a row with fewer than N
// distinct large values (bf16 logits far from zero, many at the type's lowest value)
// sends its tiles to beam_tile_slow, 2300 us for N = 32; -inf costs nothing.
template <typename T, int NV>
__global__ void __launch_bounds__(kBeamThreads, sizeof(T) == 2 ? 4 : 3)
beam_tiles_kernel(const __grid_constant__ BeamParams p) {
  constexpr int VE = 16 / sizeof(T);
  __shared__ float s_m[kBeamWarps], s_s[kBeamWarps];
  __shared__ uint32_t s_order[kBeamThreads], s_tau;
  __shared__ int s_n;
  __shared__ uint64_t s_key[kBeamBuffer], s_best[kBeamWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row = blockIdx.x / p.tiles, tile = blockIdx.x % p.tiles;
  if (tid == 0) s_n = 0;
  pdl_wait_primary();
  pdl_launch_dependents();
  if (p.finished != nullptr && p.finished[row]) return;       // its one candidate needs no logits
  const T* base = static_cast<const T*>(p.logits) + (int64_t)row * p.stride;
  const int lead = (int)((reinterpret_cast<uintptr_t>(base) & 15) / sizeof(T));
  const uint4* vec = reinterpret_cast<const uint4*>(base - lead);
  const int nvec = (lead + p.V + VE - 1) / VE;                    // aligned blocks of the row
  const int v0 = tile * (kBeamThreads * NV) + tid;
  const int64_t slot = (int64_t)row * p.tiles + tile;
  float* out_x = p.tile_x + slot * p.N;
  int32_t* out_v = p.tile_v + slot * p.N;
  const int first = tile * (kBeamThreads * NV * VE);              // the tile's first token
  uint4 raw[NV];
  if (lead == 0 && first + kBeamThreads * NV * VE <= p.V) {
#pragma unroll
    for (int j = 0; j < NV; ++j) raw[j] = __ldcs(vec + v0 + j * kBeamThreads);
  } else {
    constexpr uint32_t kNone = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int v = v0 + j * kBeamThreads;
      raw[j] = make_uint4(kNone, kNone, kNone, kNone);
      if (v < nvec) raw[j] = __ldcs(vec + v);
    }
    if (lead > 0) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int v = v0 + j * kBeamThreads + 1;
        uint4 next = make_uint4(kNone, kNone, kNone, kNone);
        if (v < nvec) next = __ldcs(vec + v);
        raw[j] = beam_shift<T>(raw[j], next, lead);
      }
    }
    // the row's last block, and those behind it, hold values of its neighbours
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int e0 = (v0 + j * kBeamThreads) * VE;
      if (e0 + VE > p.V) {
        uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          if (e0 + e >= p.V) {
            if constexpr (sizeof(T) == 4) w[e] = kNone;
            else w[e >> 1] = (e & 1) ? (w[e >> 1] & 0xffffu) | 0xff800000u : (w[e >> 1] & 0xffff0000u) | 0xff80u;
          }
        }
        raw[j] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
  float top[NV], mx = -INFINITY;                 // largest value of each block
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    top[j] = beam_block_max<T>(raw[j]);
    mx = fmaxf(mx, top[j]);
  }
  const uint32_t order = mx > -INFINITY ? beam_order(mx) : 0u;
  const float mw = warp_max(mx);
  float sum0 = 0.f, sum1 = 0.f;
  if (!beam_far(mw)) {
    const float base_w = beam_base(mw);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < VE; e += 2) {
        sum0 += ex2_approx_ftz(fmaf(beam_value<T>(raw[j], e), kBeamLog2e, -base_w));
        sum1 += ex2_approx_ftz(fmaf(beam_value<T>(raw[j], e + 1), kBeamLog2e, -base_w));
      }
  } else {
    const float mu = mw == -INFINITY ? 0.f : mw;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < VE; ++e)
        sum0 += ex2_approx_ftz((beam_value<T>(raw[j], e) - mu) * kBeamLog2e);
  }
  const float sum = warp_sum(sum0 + sum1);
  if (lane == 0) {
    s_m[warp] = mw;
    s_s[warp] = sum;
  }
  s_order[tid] = order;
  __syncthreads();
  // a bound that the largest values of N threads reach, by one warp (the bound of a
  // warp's own 32 threads lets seven times as many values through)
  if (warp == 0) {
    uint32_t x[kBeamWarps], tau = 0;
#pragma unroll
    for (int w = 0; w < kBeamWarps; ++w) x[w] = s_order[w * 32 + lane];
    for (int i = 0; i < p.N; ++i) {
      uint32_t t = x[0];
#pragma unroll
      for (int w = 1; w < kBeamWarps; ++w) t = max(t, x[w]);
      tau = __reduce_max_sync(0xffffffffu, t);
#pragma unroll
      for (int w = 0; w < kBeamWarps; ++w)
        if (x[w] == tau) x[w] = 0;
    }
    if (lane == 0) s_tau = tau;
  } else if (tid == 32) {
    float m = s_m[0], s = 0.f;
    for (int w = 1; w < kBeamWarps; ++w) m = fmaxf(m, s_m[w]);
    for (int w = 0; w < kBeamWarps; ++w) s += beam_join(s_m[w], s_s[w], m);
    p.tile_ms[slot] = make_float2(m, s);
  }
  __syncthreads();
  const uint32_t tau = s_tau;
  if (order >= tau && order > 0) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (beam_order(top[j]) >= tau) beam_push<T>(raw[j], first + (tid + j * kBeamThreads) * VE, tau, &s_n, s_key);
  }
  __syncthreads();
  const int n = s_n;
  auto store = [&](int r, uint64_t key) {
    const uint32_t o = (uint32_t)(key >> 32);
    out_x[r] = __uint_as_float(o ^ ((uint32_t)((int32_t)~o >> 31) | 0x80000000u));
    out_v[r] = (int32_t)(0xffffffffu - (uint32_t)key);
  };
  if (n <= kBeamBuffer) {
    // each candidate counts those in front of it (keys are distinct)
    for (int i = tid; i < n; i += kBeamThreads) {
      const uint64_t key = s_key[i];
      int rank = 0;
      for (int k = 0; k < n; ++k) rank += s_key[k] > key;
      if (rank < p.N) store(rank, key);
    }
    for (int r = n + tid; r < p.N; r += kBeamThreads) out_x[r] = -INFINITY;
  } else {
    beam_tile_slow<T, NV>(base, p.V, first, p.N, out_x, out_v, s_best);
  }
}

// One CTA a request: the sums of its beams' rows, then the best of all tiles'
// candidates and the finished beams.  10.5 us of the call of 49 us above: chains of
// loads and reductions over shared memory.  The bound is the N-th of a warp's 32 lanes:
// at N = 32 nearly all candidates pass it, more than the buffer holds with many beams, and
// are taken one after the other (32 of 16 beams over 131072 tokens: the call takes 819 us).
constexpr int kBeamPickBuffer = 1024;
constexpr int kBeamAhead = 2;                // candidates a thread holds from the start

__global__ void __launch_bounds__(kBeamThreads)
beam_pick_kernel(const __grid_constant__ BeamParams p) {
  __shared__ double s_add[kBeamMax];             // score - log sum exp; -inf: no candidates
  __shared__ uint8_t s_over[kBeamMax];
  __shared__ double s_sum[kBeamMax];
  __shared__ float s_top[kBeamMax];
  __shared__ uint32_t s_tau[kBeamWarps];
  __shared__ uint64_t s_key[kBeamPickBuffer];
  __shared__ uint32_t s_at[kBeamPickBuffer];
  __shared__ uint64_t s_bk[kBeamWarps];
  __shared__ uint32_t s_ba[kBeamWarps];
  __shared__ int s_n;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r = blockIdx.x;
  if (tid == 0) s_n = 0;
  pdl_wait_primary();
  pdl_launch_dependents();
  // the first candidates of this thread, and a beam's score, while the sums are joined
  const int per = p.tiles * p.N, total = p.B * per;
  float x0[kBeamAhead];
  int v0[kBeamAhead];
#pragma unroll
  for (int i = 0; i < kBeamAhead; ++i) {
    const int at = tid + i * kBeamThreads;
    x0[i] = -INFINITY;
    v0[i] = 0;
    if (at < total) {
      x0[i] = p.tile_x[(int64_t)r * total + at];
      v0[i] = p.tile_v[(int64_t)r * total + at];
    }
  }
  const float my_score = tid < p.B ? p.scores[r * p.B + tid] : 0.f;
  for (int b = warp; b < p.B; b += kBeamWarps) {
    const int row = r * p.B + b;
    // (a finished beam's sums are stale numbers that nothing uses)
    float2 ms0 = make_float2(-INFINITY, 0.f);
    if (lane < p.tiles) ms0 = p.tile_ms[(int64_t)row * p.tiles + lane];
    const bool over = p.finished != nullptr && p.finished[row];
    float m = -INFINITY;
    bool bad = false;
    double s = 0;
    if (!over) {
      for (int c = lane; c < p.tiles; c += 32) {
        const float2 ms = c < 32 ? ms0 : p.tile_ms[(int64_t)row * p.tiles + c];
        m = fmaxf(m, ms.x);
        bad |= !(ms.x < INFINITY) || !(ms.y < INFINITY);
      }
      m = warp_max(m);
      bad = __any_sync(0xffffffffu, bad);
      for (int c = lane; c < p.tiles; c += 32) {
        const float2 ms = c < 32 ? ms0 : p.tile_ms[(int64_t)row * p.tiles + c];
        if (!bad) s += (double)beam_join(ms.x, ms.y, m);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (bad && lane == 0) record_error(PKV_DEVERR_BEAM);
    }
    if (lane == 0) {
      s_over[b] = over;
      s_top[b] = bad ? -INFINITY : m;
      s_sum[b] = s;
    }
  }
  __syncthreads();
  // one lane a beam: 64-bit logarithms are slow, one after the other even more so
  if (tid < p.B) {
    const float score = my_score, m = s_top[tid];
    double add = -INFINITY;
    if (s_over[tid]) {
      add = (double)score;
    } else if (m > -INFINITY) {
      // 2^(x c) with the float32 c is exp(x (1 + e)): e m comes off, what weighs is
      // within a few units of m
      constexpr double kLn2 = 0.69314718055994530942, kE = (double)kBeamLog2e * kLn2 - 1.;
      const double base = beam_far(m) ? (double)m : (double)beam_base(m) * kLn2 - kE * (double)m;
      add = (double)score - (base + log(s_sum[tid]));
    }
    s_add[tid] = add;
  }
  __syncthreads();
  // candidate i: beam, tile and place; a finished beam has one, its end token
  auto load = [&](int i, uint64_t& key, uint32_t& at) -> bool {
    const int b = i / per, j = i - b * per;
    const double add = s_add[b];
    double c;
    int v;
    if (s_over[b]) {
      if (j != 0) return false;
      c = add;
      v = p.eos;
    } else {
      float x;
      if (i < kBeamAhead * kBeamThreads) {
        x = i < kBeamThreads ? x0[0] : x0[1];
        v = i < kBeamThreads ? v0[0] : v0[1];
      } else {
        x = p.tile_x[(int64_t)r * total + i];
        v = p.tile_v[(int64_t)r * total + i];
      }
      if (!(x > -INFINITY)) return false;
      c = (double)x + add;
    }
    key = beam_order(c);
    at = (uint32_t)(b * p.V + v);
    return key != 0;
  };
  uint64_t key0[kBeamAhead];
  uint32_t at0[kBeamAhead];
#pragma unroll
  for (int i = 0; i < kBeamAhead; ++i) {
    at0[i] = 0;
    if (tid + i * kBeamThreads >= total || !load(tid + i * kBeamThreads, key0[i], at0[i])) key0[i] = 0;
  }
  // bound on the upper halves of the keys: N threads' largest are at or above it
  uint32_t tau = 0;
  {
    uint32_t mx = 0;
    uint64_t key;
    uint32_t at;
#pragma unroll
    for (int i = 0; i < kBeamAhead; ++i) mx = max(mx, (uint32_t)(key0[i] >> 32));
    for (int i = tid + kBeamAhead * kBeamThreads; i < total; i += kBeamThreads)
      if (load(i, key, at)) mx = (uint32_t)(key >> 32) > mx ? (uint32_t)(key >> 32) : mx;
    mx = warp_bound(mx, p.N);
    if (lane == 0) s_tau[warp] = mx;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kBeamWarps; ++w) tau = s_tau[w] > tau ? s_tau[w] : tau;
  }
  auto push = [&](uint64_t key, uint32_t at) {
    const int k = atomicAdd(&s_n, 1);
    if (k < kBeamPickBuffer) {
      s_key[k] = key;
      s_at[k] = at;
    }
  };
#pragma unroll
  for (int i = 0; i < kBeamAhead; ++i)
    if (key0[i] != 0 && (uint32_t)(key0[i] >> 32) >= tau) push(key0[i], at0[i]);
  for (int i = tid + kBeamAhead * kBeamThreads; i < total; i += kBeamThreads) {
    uint64_t key;
    uint32_t at;
    if (load(i, key, at) && (uint32_t)(key >> 32) >= tau) push(key, at);
  }
  __syncthreads();
  const int n = s_n;
  auto store = [&](int k, uint64_t key, uint32_t at) {
    const double c = __longlong_as_double(
        (long long)(key ^ ((uint64_t)((int64_t)~key >> 63) | 0x8000000000000000ull)));
    const int b = (int)(at / (uint32_t)p.V), v = (int)(at - (uint32_t)b * (uint32_t)p.V);
    const int64_t o = (int64_t)r * p.N + k;
    p.tokens[o] = v;
    p.parents[o] = b;
    p.scores_out[o] = (float)c;
    if (p.finished_out != nullptr) p.finished_out[o] = s_over[b] || v == p.eos;
  };
  if (n <= kBeamPickBuffer) {
    for (int i = tid; i < n; i += kBeamThreads) {
      const uint64_t key = s_key[i];
      const uint32_t at = s_at[i];
      int rank = 0;
      for (int k = 0; k < n; ++k) rank += s_key[k] > key || (s_key[k] == key && s_at[k] < at);
      if (rank < p.N) store(rank, key, at);
    }
  } else {
    // very many equal candidates (beams alike): one after the other
    uint64_t last_key = ~0ull;
    uint32_t last_at = 0;
    for (int k = 0; k < p.N; ++k) {
      uint64_t bk = 0;
      uint32_t ba = 0xffffffffu;
      for (int i = tid; i < total; i += kBeamThreads) {
        uint64_t key;
        uint32_t at;
        if (!load(i, key, at)) continue;
        const bool behind = key < last_key || (key == last_key && at > last_at);
        if (behind && (key > bk || (key == bk && at < ba))) {
          bk = key;
          ba = at;
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const uint64_t yk = __shfl_xor_sync(0xffffffffu, bk, o);
        const uint32_t ya = __shfl_xor_sync(0xffffffffu, ba, o);
        if (yk > bk || (yk == bk && ya < ba)) {
          bk = yk;
          ba = ya;
        }
      }
      __syncthreads();
      if (lane == 0) {
        s_bk[warp] = bk;
        s_ba[warp] = ba;
      }
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kBeamWarps; ++w)
        if (s_bk[w] > bk || (s_bk[w] == bk && s_ba[w] < ba)) {
          bk = s_bk[w];
          ba = s_ba[w];
        }
      last_key = bk;
      last_at = ba;
      if (tid == 0) store(k, bk, ba);             // (more than kBeamPickBuffer: there are N)
    }
  }
  for (int k = n + tid; k < p.N; k += kBeamThreads) {
    const int64_t o = (int64_t)r * p.N + k;
    p.tokens[o] = -1;
    p.parents[o] = -1;
    p.scores_out[o] = -INFINITY;
    if (p.finished_out != nullptr) p.finished_out[o] = 1;
  }
}

}  // namespace pkv
