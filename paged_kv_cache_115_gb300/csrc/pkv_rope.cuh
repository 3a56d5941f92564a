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
// Called by W warps that `sync` makes wait for one another.
template <int W, typename Sync>
__device__ __forceinline__ void rope_int8_rows(const RopeParams& p, int64_t slot,
                                               int64_t pool_row, const float (&amax)[2],
                                               const float* s_all, float (*s_amax)[W],
                                               Sync&& sync) {
  if (slot < 0) return;
  const int n = p.H_kv * p.D;
#pragma unroll
  for (int z = 0; z < 2; ++z) {
    const float m = warp_max(amax[z]);
    if ((threadIdx.x & 31) == 0) s_amax[z][threadIdx.x >> 5] = m;
  }
  sync();
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
// row in shared memory (a rotated pair may sit in two lanes).  Bound by its
// instructions, a value at a time: 16381 tokens of 32 + 2 x 8 heads take 239 us
// at head_dim 80 (1.1 TB/s), 251 at 96, 365 at 112, and 286 at 128 in rows off
// 16-byte boundaries.
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
  if constexpr (FMT == 2) rope_int8_rows<W>(p, slot, pool_row, amax, s_all, s_amax, [] { __syncthreads(); });
}

// Ring form: head_dim 64 or 128 (256 for bf16), rows and strides on 16-byte
// boundaries, the rotation a multiple of 8 values (4 for float32).  Persistent
// CTAs; a producer warp brings whole tokens (query, key and value heads, and
// the position's cosines and sines) into a ring of shared-memory stages by
// bulk copies, so that the bytes in flight do not hang on registers; eight
// warps compute.  A lane holds V = 16 / sizeof(TIN) values of a row, V / 2
// from either half of the rotation (interleaved: neighbours; behind the
// rotation: as they come), so that a rotated pair sits in one lane and needs
// no shuffle; a row takes D / V lanes, a CTA 256 V / D rows at once.
// Bound by HBM: 2 (H_q + 2 H_kv) D e bytes a token; 16381 tokens of 32 + 2 x 8
// heads of 128 with norms: bf16 pools 68 us (65 without norms), bf16 K + FP8 V
// 69, FP8 73, float32 131 (6.2 TB/s).  INT8 120: a token's scale needs its whole
// row, kept in shared memory and read again behind two barriers.
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

// N values (half of a lane's) as T, and as e4m3 codes of x / scale.
template <typename T, int N>
__device__ __forceinline__ void rope_store_half(T* dst, const float* x) {
  if constexpr (sizeof(T) == 4) {
    static_assert(N == 2, "8 bytes");
    *reinterpret_cast<float2*>(dst) = make_float2(x[0], x[1]);
  } else if constexpr (N == 4) {
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
  } else {
    *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(x[0], x[1]);
  }
}
template <int N>
__device__ __forceinline__ void rope_store_codes(uint8_t* dst, const float* x, float scale) {
  uint32_t w[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; ++i)
    w[i] = __nv_cvt_float2_to_fp8x2(
        make_float2(__fdiv_rn(x[2 * i], scale), __fdiv_rn(x[2 * i + 1], scale)), __NV_SATFINITE,
        __NV_E4M3);
  if constexpr (N == 4) *reinterpret_cast<uint32_t*>(dst) = w[0] | (w[1] << 16);
  else *reinterpret_cast<uint16_t*>(dst) = (uint16_t)w[0];
}
template <typename TIN, int FMT>
struct RopeKType { using T = TIN; };
template <typename TIN>
struct RopeKType<TIN, 3> { using T = __nv_bfloat16; };

// 1-D bulk copy with an L2 hint for data that is read once.
__device__ __forceinline__ void bulk_load_hint(uint32_t dst, const void* src, uint32_t bytes,
                                               uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
      "[%0], [%1], %2, [%3], %4;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar), "l"(policy)
      : "memory");
}

constexpr int kRopeRingThreads = kRopeThreads + 32;
// Two stages in each of three CTAs an SM: more bytes in flight make reads and
// writes worse neighbours in HBM.  16381 tokens of 32 + 2 x 8 heads of 128,
// 411 MB: 65.4 us (6.3 TB/s); three and four stages 69.7 and 71.5, four CTAs
// with two to four stages 70.4, 73.3, 72.9, two CTAs with four 74.1.
constexpr int kRopeStages = 2;
constexpr int kRopeCtas = 3;

// V / 2 values (8 bytes) at a time.
template <typename TIN>
__device__ __forceinline__ void rope_unpack2(uint2 a, uint2 b, float (&x)[16 / sizeof(TIN)]) {
  rope_unpack<TIN>(make_uint4(a.x, a.y, b.x, b.y), x);
}

template <typename TIN, int FMT, int D, bool PAIRS>
__global__ void __launch_bounds__(kRopeRingThreads, kRopeCtas)
rope_ring_kernel(const __grid_constant__ RopeParams p, int stage_bytes) {
  constexpr int stages = kRopeStages;
  constexpr int V = 16 / sizeof(TIN), HV = V / 2, LANES = D / V, RPI = kRopeThreads / LANES;
  static_assert(LANES <= 32, "a row must fit a warp");
  constexpr int W = kRopeThreads / 32;
  extern __shared__ __align__(128) uint8_t s_ring[];
  __shared__ __align__(8) uint64_t s_full[kRopeStages], s_empty[kRopeStages];
  __shared__ long long s_slot[kRopeStages];
  __shared__ int s_token[kRopeStages];
  __shared__ float s_amax[2][W];
  float* const s_all = reinterpret_cast<float*>(s_ring + (size_t)stages * stage_bytes);   // INT8
  // the consumers among themselves
  auto sync = [] { asm volatile("bar.sync 1, %0;" ::"n"(kRopeThreads) : "memory"); };
  auto all_of = [](bool ok) -> bool {
    uint32_t all;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\tbar.red.and.pred q, 1, %1, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(all)
        : "n"(kRopeThreads), "r"((uint32_t)ok)
        : "memory");
    return all != 0;
  };
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int q_bytes = p.H_q * D * (int)sizeof(TIN), kv_bytes = p.H_kv * D * (int)sizeof(TIN);
  if (tid == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(smem_u32(&s_full[i]), 1);
      mbar_init(smem_u32(&s_empty[i]), W);
    }
    fence_barrier_init();
  }
  __syncthreads();
  pdl_wait_primary();
  pdl_launch_dependents();

  if (warp == W) {
    // =================== producer ===================
    const uint64_t policy = l2_policy_evict_first();
    int n = 0;                                          // stages filled
    bool ok = true;
    for (int t0 = blockIdx.x; t0 < p.T && ok; t0 += 32 * gridDim.x) {
      // positions and slots of the CTA's next 32 tokens
      const int tl = t0 + lane * (int)gridDim.x;
      int pos = -1;
      long long slot = -1;
      if (tl < p.T) {
        pos = p.positions[tl];
        slot = p.slots[tl];
        if (pos >= p.max_pos) {
          record_error(PKV_DEVERR_POSITION);
          pos = -1;
        } else if (pos >= 0 && (slot < 0 || slot >= p.num_slots)) {
          if (slot != -1) record_error(PKV_DEVERR_SLOT);
          slot = -1;
        }
      }
      unsigned todo = __ballot_sync(0xffffffffu, pos >= 0);           // the others are skipped
      while (todo) {
        const int l = __ffs(todo) - 1;
        todo &= todo - 1;
        const int t = t0 + l * (int)gridDim.x;
        const int pt = __shfl_sync(0xffffffffu, pos, l);
        const long long st = __shfl_sync(0xffffffffu, slot, l);
        const int stage = n % stages;
        ok = __all_sync(0xffffffffu,
                        mbar_wait_bounded(smem_u32(&s_empty[stage]), ((n / stages) & 1) ^ 1));
        if (!ok) break;
        if (lane == 0) {
          const uint32_t full = smem_u32(&s_full[stage]);
          const uint32_t dst = smem_u32(s_ring + (size_t)stage * stage_bytes);
          s_slot[stage] = st;
          s_token[stage] = t;
          mbar_arrive_expect_tx(full, q_bytes + 2 * kv_bytes + 4 * p.rot);
          bulk_load_hint(dst, static_cast<const TIN*>(p.q) + t * p.q_stride, q_bytes, full, policy);
          bulk_load_hint(dst + q_bytes, static_cast<const TIN*>(p.k) + t * p.k_stride, kv_bytes, full, policy);
          bulk_load_hint(dst + q_bytes + kv_bytes, static_cast<const TIN*>(p.v) + t * p.v_stride, kv_bytes, full, policy);
          if (p.rot > 0)
            bulk_load(dst + q_bytes + 2 * kv_bytes, p.cos_sin + (int64_t)pt * p.rot, 4 * p.rot, full);
        }
        __syncwarp();
        ++n;
      }
    }
    // the consumers' end: a stage without a token
    const int end = n % stages;
    ok = ok && __all_sync(0xffffffffu,
                          mbar_wait_bounded(smem_u32(&s_empty[end]), ((n / stages) & 1) ^ 1));
    if (ok) {
      if (lane == 0) {
        s_slot[end] = -2;
        mbar_arrive(smem_u32(&s_full[end]));
      }
    } else {
      if (lane == 0) record_error(PKV_DEVERR_TIMEOUT);
      // do not leave the CTA while our own copies may still land
      for (int i = max(0, n - stages); i < n; ++i)
        mbar_wait_bounded(smem_u32(&s_full[i % stages]), (i / stages) & 1);
    }
    return;
  }

  // =================== consumers ===================
  const int li = tid % LANES;
  const int half = p.rot >> 1;
  // this lane's values: HV from ea on, HV from eb on
  const bool turned = li * V < p.rot;
  const int ea = PAIRS || !turned ? li * V : li * HV;
  const int eb = PAIRS || !turned ? ea + HV : half + li * HV;
  uint2 wqa = make_uint2(0, 0), wqb = wqa, wka = wqa, wkb = wqa;
  if (p.wq != nullptr) {
    wqa = __ldg(reinterpret_cast<const uint2*>(static_cast<const TIN*>(p.wq) + ea));
    wqb = __ldg(reinterpret_cast<const uint2*>(static_cast<const TIN*>(p.wq) + eb));
  }
  if (p.wk != nullptr) {
    wka = __ldg(reinterpret_cast<const uint2*>(static_cast<const TIN*>(p.wk) + ea));
    wkb = __ldg(reinterpret_cast<const uint2*>(static_cast<const TIN*>(p.wk) + eb));
  }
  // rows of this warp in a group of RPI: row0 + sub
  const int row0 = warp * (32 / LANES), sub = lane / LANES;
  int stage = 0, round = 0;
  for (;;) {
    bool ok = __all_sync(0xffffffffu, mbar_wait_bounded(smem_u32(&s_full[stage]), round & 1));
    // INT8: the warps wait for one another below, so they give up together
    if constexpr (FMT == 2) ok = all_of(ok);
    if (!ok) {
      if (lane == 0) record_error(PKV_DEVERR_TIMEOUT);
      return;
    }
    uint8_t* sb = s_ring + (size_t)stage * stage_bytes;
    const long long slot = s_slot[stage];
    if (slot == -2) return;
    const int t = s_token[stage];
    float c[HV], s[HV];
#pragma unroll
    for (int i = 0; i < HV; ++i) {
      c[i] = 1.f;
      s[i] = 0.f;
    }
    if (turned) {
      const float* cs = reinterpret_cast<const float*>(sb + q_bytes + 2 * kv_bytes) + li * HV;
#pragma unroll
      for (int i = 0; i < HV; ++i) {
        c[i] = cs[i];
        s[i] = cs[half + i];
      }
    }
    const TIN* const src = reinterpret_cast<const TIN*>(sb);      // q, k and v rows one after the other
    const int64_t pool_row = slot * p.H_kv * D;
    float amax[2] = {0.f, 0.f};
    // a head row of this lane: norm (weights not null) and rotation
    auto turn = [&](uint2 xa, uint2 xb, const void* weight, uint2 wa, uint2 wb, float (&y)[V]) {
      float x[V];
      rope_unpack2<TIN>(xa, xb, x);
      if (weight != nullptr) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        float w[V];
        rope_unpack2<TIN>(wa, wb, w);
        const float inv = rsqrtf(ss / D + p.eps);
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] *= inv * w[i];
      }
      if constexpr (PAIRS) {
#pragma unroll
        for (int i = 0; i < HV; ++i) {
          y[2 * i] = x[2 * i] * c[i] - x[2 * i + 1] * s[i];
          y[2 * i + 1] = x[2 * i + 1] * c[i] + x[2 * i] * s[i];
        }
      } else {
        // two pairs at a time as packed float32 operations
#pragma unroll
        for (int i = 0; i < HV; i += 2) {
          const float2 a = make_float2(x[i], x[i + 1]), b = make_float2(x[HV + i], x[HV + i + 1]);
          const float2 c2 = make_float2(c[i], c[i + 1]), s2 = make_float2(s[i], s[i + 1]);
          const float2 lo = __ffma2_rn(b, make_float2(-s2.x, -s2.y), __fmul2_rn(a, c2));
          const float2 hi = __ffma2_rn(a, s2, __fmul2_rn(b, c2));
          y[i] = lo.x; y[i + 1] = lo.y;
          y[HV + i] = hi.x; y[HV + i + 1] = hi.y;
        }
      }
      // behind the rotation values stay: turned by 0 they would meet 0 x inf
      // of one another, and a zero could lose its sign (p.rot: one branch for
      // all where everything turns; 64 tokens 2.7 us, 2.9 without it)
      if (p.rot < D && !turned) {
#pragma unroll
        for (int i = 0; i < V; ++i) y[i] = x[i];
      }
    };
    // rows of a kind for this warp: `row0` is the same for a whole warp, so
    // that shuffles stay whole; lanes of a row past the last one repeat it
    TIN* qo = static_cast<TIN*>(p.q_out) + t * p.qo_stride;
#pragma unroll 4
    for (int r0 = row0; r0 < p.H_q; r0 += RPI) {
      const int r = min(r0 + sub, p.H_q - 1) * D;
      float y[V];
      turn(*reinterpret_cast<const uint2*>(src + r + ea), *reinterpret_cast<const uint2*>(src + r + eb),
           p.wq, wqa, wqb, y);
      const uint4 o = rope_pack<TIN>(y);
      *reinterpret_cast<uint2*>(qo + r + ea) = make_uint2(o.x, o.y);
      *reinterpret_cast<uint2*>(qo + r + eb) = make_uint2(o.z, o.w);
    }
    if (slot >= 0) {                                      // else the pools are left alone
      const TIN* const ks = src + p.H_q * D;
      const TIN* const vs = ks + p.H_kv * D;
      for (int r0 = row0; r0 < p.H_kv; r0 += RPI) {
        const int r = min(r0 + sub, p.H_kv - 1) * D;
        float y[V];
        turn(*reinterpret_cast<const uint2*>(ks + r + ea), *reinterpret_cast<const uint2*>(ks + r + eb),
             p.wk, wka, wkb, y);
        if constexpr (FMT == 2) {
          float* dst = s_all + r;
#pragma unroll
          for (int i = 0; i < HV; ++i) {
            dst[ea + i] = y[i];
            dst[eb + i] = y[i + HV];
            amax[0] = fmaxf(amax[0], fmaxf(fabsf(y[i]), fabsf(y[i + HV])));
          }
        } else if constexpr (FMT == 1) {
          rope_store_codes<HV>(p.k_cache + pool_row + r + ea, y, p.k_scale);
          rope_store_codes<HV>(p.k_cache + pool_row + r + eb, y + HV, p.k_scale);
        } else {
          using TK = typename RopeKType<TIN, FMT>::T;
          TK* dst = reinterpret_cast<TK*>(p.k_cache) + pool_row + r;
          rope_store_half<TK, HV>(dst + ea, y);
          rope_store_half<TK, HV>(dst + eb, y + HV);
        }
      }
      // value rows on the other half of the warps first
      for (int r0 = (row0 + RPI / 2) % RPI; r0 < p.H_kv; r0 += RPI) {
        const int r = min(r0 + sub, p.H_kv - 1) * D;
        const uint4 raw = *reinterpret_cast<const uint4*>(vs + r + li * V);
        if constexpr (FMT == 0) {
          *reinterpret_cast<uint4*>(reinterpret_cast<TIN*>(p.v_cache) + pool_row + r + li * V) = raw;
        } else {
          float x[V];
          rope_unpack<TIN>(raw, x);
          if constexpr (FMT == 2) {
            float* dst = s_all + p.H_kv * D + r + li * V;
#pragma unroll
            for (int i = 0; i < V; ++i) {
              dst[i] = x[i];
              amax[1] = fmaxf(amax[1], fabsf(x[i]));
            }
          } else {
            rope_store_codes<HV>(p.v_cache + pool_row + r + li * V, x, p.v_scale);
            rope_store_codes<HV>(p.v_cache + pool_row + r + li * V + HV, x + HV, p.v_scale);
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&s_empty[stage]));
    if (++stage == stages) {
      stage = 0;
      ++round;
    }
    if constexpr (FMT == 2) {
      rope_int8_rows<W>(p, slot, pool_row, amax, s_all, s_amax, sync);
      sync();                                           // s_all is free for the next token
    }
  }
}

}  // namespace pkv
