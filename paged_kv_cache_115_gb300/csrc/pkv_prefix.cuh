// Decode attention over a prefix that the whole batch shares and each
// sequence's own tokens behind it.
//
//   out = softmax over (prefix keys, own keys) . V, as partial states
//   (m, l, o) of both parts merged by M = max m, l = sum l 2^(m - M),
//   out = sum o 2^(m - M) / l.
//
// The prefix part is one matrix product over the query rows of the whole
// batch: row r of KV head j is head j G + r % G of token r / G, and tiles of
// 128 rows meet every prefix key once (tcgen05).  The own part is the
// stream-K decode kernel on the tokens from prefix_len on.  The first is bound
// by the tensor cores (or, with one tile of rows, by HBM), the second by HBM;
// they run side by side on disjoint SMs: the prefix kernel releases its
// dependent launch at once, the decode kernel does not wait for it, and both
// derive from the lengths on the device how many of the SMs each takes.  The
// merge waits for both.
#pragma once

#include "pkv_attention_tc.cuh"
#include "pkv_prefill_tc05.cuh"

namespace pkv {

constexpr int kPxBN = 64;             // keys per step
constexpr int kPxKStages = 5;
constexpr int kPxVStages = 5;
constexpr int kPxThreads = 384;

struct PxParams {
  CUtensorMap tmap_k;
  CUtensorMap tmap_v;
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  const int32_t* prefix_table;
  const int32_t* cu;                  // null: one query row per sequence
  const int32_t* lens;
  PxSplit split;                      // how the SMs are shared with the decode kernel
  int2* items;                        // {first CTA, CTAs} of each item, for the merge
  const int4* meta;                   // own part: {first slot, partials, 0, 0} of each token
  const float2* own_ml;               // own part: [slot][H_q]
  const float* own_o;
  float2* ml;                         // prefix part: [CTA + item][rows of an item]
  float* o;
  long long num_blocks;
  long long own_slots;
  int own_stride;                     // slots between the partials of a token
  int max_len, row_tokens;            // bounds of a length
  int S, T, H_q, H_kv, G, block_size;
  float scale_log2;
};

template <int D>
struct PxCfg {
  static constexpr int NH = D / 64;
  static constexpr int QHALF = kT5Rows * 128;             // 16 KiB
  static constexpr int QBYTES = NH * QHALF;               // one query tile
  static constexpr int KVHALF = kPxBN * 128;              // 8 KiB
  static constexpr int KBYTES = NH * KVHALF;              // one K (or V) tile
  static constexpr int NBOX = NH * (kPxBN / 16);
  static constexpr int Q_OFF = 0;                         // [tile][half]
  static constexpr int K_OFF = 2 * QBYTES;
  static constexpr int V_OFF = K_OFF + kPxKStages * KBYTES;
  static constexpr int BAR_OFF = V_OFF + kPxVStages * KBYTES;
  // k_full/k_empty[KS], v_full/v_empty[VS], per tile: s_full[2], p_free[2],
  // p_full[2], o_done, q_full; mma_idle
  static constexpr int NBAR = 2 * (kPxKStages + kPxVStages) + 2 * 8 + 1;
  static constexpr int SLOT_OFF = BAR_OFF + 8 * NBAR;
  static constexpr int SMEM = SLOT_OFF + 16 + 1024;
  // per tile: S buffers 0, 1 (64 columns each: fp32 S, then P as bf16 pairs
  // in the lower 32), O (128)
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t IDESC_QK = umma_idesc_bf16(kT5Rows, kPxBN, 0, 0);
  static constexpr uint32_t IDESC_PV = umma_idesc_bf16(kT5Rows, D, 0, 1);
};

// Query rows of the launch: token count times G (0 .. T G).
__device__ __forceinline__ int px_tokens(const int32_t* cu, int S, int T) {
  if (cu == nullptr) return S;
  const int t = cu[S];
  return t < 0 ? 0 : min(t, T);
}

// Sequence of packed token t and whether it is consistent: cu[s] <= t <
// cu[s+1] <= T and n <= its length; L its clamped length, i its index.
__device__ __forceinline__ bool px_row(const PxParams& p, int t, int& s, int& i, int& n, int& L) {
  s = t;
  i = 0;
  n = 1;
  if (p.cu != nullptr) {
    int lo = 0, hi = p.S;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.cu[mid] <= t) lo = mid; else hi = mid;
    }
    s = lo;
    const int c0 = p.cu[s], c1 = p.cu[s + 1];
    i = t - c0;
    n = c1 - c0;
    if (i < 0 || t >= c1 || c0 < 0 || c1 > p.T || n > p.split.max_q) return false;
  }
  const int cap = min(p.max_len, p.row_tokens);
  L = max(0, min(p.lens[s], cap));
  return p.cu == nullptr || n <= L;
}

// One lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(p));
  return p != 0;
}

// 64 consecutive fp32 columns of this thread's TMEM lane, landed.
__device__ __forceinline__ void tmem_ld64_wait(uint32_t taddr, float (&v)[64]) {
  uint32_t a[32], b[32];
  tmem_ld32(taddr, a);
  tmem_ld32(taddr + 32, b);
  tmem_wait_ld();
#pragma unroll
  for (int e = 0; e < 32; ++e) {
    v[e] = __uint_as_float(a[e]);
    v[32 + e] = __uint_as_float(b[e]);
  }
}

// ===========================================================================
// Prefix part.  Item = (KV head, pair of 128-row tiles; SOLO: one tile); an
// item takes ceil(prefix_len / 64) steps of 64 keys.  CTA c of n1 owns steps
// [c S / n1, (c + 1) S / n1) of all S: a run of one item's steps is one
// partial state, in slot c + item (distinct, as in the decode kernel).
//
// Warps 0-3: softmax of tile A, 4-7: of tile B (one thread per query row =
// TMEM lane); warp 8: TMA producer of K tiles, warp 10: of V tiles; warp 9:
// TMEM and, on one lane, S = Q K^T for both tiles (two S buffers each); warp
// 11, one lane: O += P V.  P overwrites the S buffer it came from and is read
// from TMEM as the A operand.
// P is rounded to bf16 (to nearest): the tensor cores take both operands of
// a product in one type, and V is bf16.  The relative error of a weight is at
// most 2^-8 and independent from key to key, below the rounding of the
// output; the row sum l adds the unrounded weights in fp32.
// The exponent base of a row is raised only when its maximum grows by more
// than 2^8, so O is rescaled in TMEM rarely.  Every wait is bounded.
// ===========================================================================
template <int D, bool SOLO>
__global__ void __launch_bounds__(kPxThreads, 1)
prefix_tc05_kernel(const __grid_constant__ PxParams p) {
  using C = PxCfg<D>;
  constexpr int NT = SOLO ? 1 : 2;                        // query tiles per item
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ long long s_chunks[kPxThreads / 32];
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bars = sbase + C::BAR_OFF;
  const uint32_t k_full = bars, k_empty = k_full + 8 * kPxKStages;
  const uint32_t v_full = k_empty + 8 * kPxKStages, v_empty = v_full + 8 * kPxVStages;
  const uint32_t tb0 = v_empty + 8 * kPxVStages;          // per-tile barriers, 8 each
  auto s_full = [&](int x, int b) { return tb0 + 64 * x + 8 * b; };
  auto p_free = [&](int x, int b) { return tb0 + 64 * x + 16 + 8 * b; };
  auto p_full = [&](int x, int b) { return tb0 + 64 * x + 32 + 8 * b; };
  auto o_done = [&](int x) { return tb0 + 64 * x + 48; };
  auto q_full = [&](int x) { return tb0 + 64 * x + 56; };
  const uint32_t mma_idle = tb0 + 128;
  uint32_t* slot = reinterpret_cast<uint32_t*>(smem + C::SLOT_OFF);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x;

  // ---- the SMs of this part: everything the kernel in front wrote is there
  // after the wait, for the decode kernel too
  pdl_wait_primary();
  pdl_launch_dependents();
  long long chunks = 0;
  for (int s = tid; s < p.S; s += kPxThreads)
    chunks += px_own_chunks(p.split, p.cu, p.T, s, max(0, min(p.lens[s], min(p.max_len, p.row_tokens))));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) chunks += __shfl_xor_sync(0xffffffffu, chunks, o);
  if (lane == 0) s_chunks[warp] = chunks;
  __syncthreads();
  chunks = 0;
#pragma unroll
  for (int w = 0; w < kPxThreads / 32; ++w) chunks += s_chunks[w];
  const int R = px_tokens(p.cu, p.S, p.T) * p.G;           // query rows per KV head
  const int npairs = (R + NT * kT5Rows - 1) / (NT * kT5Rows);
  const int P = p.split.prefix_len;
  const int nkt = (P + kPxBN - 1) / kPxBN;
  const long long steps = (long long)npairs * p.H_kv * nkt;
  const int n1 = px_ctas(p.split, steps, chunks);
  if (cta >= n1) return;
  if (cta == n1 - 1) {                                     // which CTAs hold steps of each item
    for (int x = tid; x < npairs * p.H_kv; x += kPxThreads) {
      const int a = cta_of_chunk((long long)x * nkt, steps, n1);
      p.items[x] = make_int2(a, cta_of_chunk((long long)(x + 1) * nkt - 1, steps, n1) - a + 1);
    }
  }
  const long long g0 = cta * steps / n1;
  const int ng = (int)((cta + 1) * steps / n1 - g0);       // steps of this CTA

  if (tid == 0) {
    for (int i = 0; i < kPxKStages; ++i) {
      mbar_init(k_full + 8 * i, 1);
      mbar_init(k_empty + 8 * i, NT);                      // every tile's S reads K
    }
    for (int i = 0; i < kPxVStages; ++i) {
      mbar_init(v_full + 8 * i, 1);
      mbar_init(v_empty + 8 * i, 1);
    }
    for (int x = 0; x < 2; ++x) {
      for (int b = 0; b < 2; ++b) {
        mbar_init(s_full(x, b), 1);
        mbar_init(p_free(x, b), 1);
        mbar_init(p_full(x, b), kT5Rows);
      }
      mbar_init(o_done(x), 1);
      mbar_init(q_full(x), kT5Rows);
    }
    mbar_init(mma_idle, 2);
    fence_barrier_init();
  }
  if (warp == 9) tmem_alloc(smem_u32(slot), C::TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;
  const int K = p.block_size;

  if (warp == 8 || warp == 10) {
    // =================== TMA producers: warp 8 K tiles, warp 10 V tiles ===================
    const int kv = warp == 10;
    const CUtensorMap* map = kv ? &p.tmap_v : &p.tmap_k;
    const int NS = kv ? kPxVStages : kPxKStages;
    const uint32_t full = kv ? v_full : k_full, empty = kv ? v_empty : k_empty;
    uint8_t* ring = smem + (kv ? C::V_OFF : C::K_OFF);
    if (lane == 0) prefetch_tensormap(map);
    // the prefix is read once per pair of tiles: kept in L2 when there are several
    const uint64_t policy = npairs > 1 ? l2_policy_evict_normal() : l2_policy_evict_first();
    const int sbl = K < 16 ? 1 : 0;                       // 8-token blocks: 8-row boxes
    const int ncopy = C::NBOX << sbl;                     // <= 16: one box per lane
    const int bi = lane >> sbl, u = lane & sbl;
    const int half = bi >> 2, rb = bi & 3;
    const int tr = rb * 16 + (u << 3);
    int kt = (int)(g0 % nkt), j = (int)(g0 / nkt / npairs);
    int left = (int)(((long long)(j + 1) * npairs * nkt) - g0);     // steps left of KV head j
    // the table entry of this lane's box, loaded one step ahead
    auto table_entry = [&](int g, int t) -> long long {
      const int tok = t * kPxBN + tr;
      if (lane >= ncopy || g >= ng || tok >= P) return -1;
      return p.prefix_table[tok / K];
    };
    long long phys_next = table_entry(0, kt);
    int g = 0;
    bool ok = true;
    for (; g < ng; ++g) {
      const int stage = g % NS;
      const long long phys = phys_next;
      const int ktn = kt + 1 == nkt ? 0 : kt + 1;
      phys_next = table_entry(g + 1, ktn);
      if (!mbar_wait_bounded(empty + 8 * stage, ((g / NS) & 1) ^ 1)) {
        record_error(PKV_DEVERR_TIMEOUT);
        ok = false;
        break;
      }
      if (lane == 0) mbar_arrive_expect_tx(full + 8 * stage, C::KBYTES);
      __syncwarp();
      if (lane < ncopy) {
        const int tok = kt * kPxBN + tr;
        int row = -32;                                    // past the prefix: zero fill
        if (tok < P) {
          if (phys < 0 || phys >= p.num_blocks) {
            record_error(PKV_DEVERR_BLOCK_ID);
          } else {
            row = (int)(phys * K + (tok - (tok / K) * K));
          }
        }
        tma_load_3d(smem_u32(ring + stage * C::KBYTES + half * C::KVHALF + tr * 128), map,
                    full + 8 * stage, half * 64, j, row, policy);
      }
      __syncwarp();
      kt = ktn;
      if (--left == 0) {
        ++j;
        left = npairs * nkt;
      }
    }
    if (!ok) {
      for (int kk = max(0, g - NS); kk < g; ++kk)
        mbar_wait_bounded(full + 8 * (kk % NS), (kk / NS) & 1);
    }
  } else if (warp == 9 || warp == 11) {
    // =================== MMA issue: warp 9 S = Q K^T, warp 11 O += P V ===================
    // The whole warp walks the loop and one elected lane issues: under a lane
    // test the compiler cannot tell that the descriptors are uniform, and an
    // MMA took 80 to 90 cycles to issue.
    bool ok = true;
    int kt = (int)(g0 % nkt), seg = 0;
    for (int g = 0; g < ng && ok; ++g) {
      const bool first = g == 0 || kt == 0;                // of a segment
      if (warp == 9) {
        const int stage = g % kPxKStages, b = g & 1;
        if (first) {
          for (int x = 0; x < NT && ok; ++x) ok = mbar_wait_bounded(q_full(x), seg & 1);
          ++seg;
        }
        ok = ok && mbar_wait_bounded(k_full + 8 * stage, (g / kPxKStages) & 1);
        const uint32_t kb = sbase + C::K_OFF + stage * C::KBYTES;
        for (int x = 0; x < NT && ok; ++x) {
          // S buffer b of tile x holds P(g - 2) until O += P(g - 2) V is done
          ok = __all_sync(0xffffffffu,
                          g < 2 || mbar_wait_bounded(p_free(x, b), ((g >> 1) - 1) & 1));
          if (!ok) break;
          tc_fence_after();
          const uint32_t qb = sbase + C::Q_OFF + x * C::QBYTES;
          const uint32_t sd = tmem + x * 256 + b * kPxBN;
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint64_t ad = umma_desc_sw128(qb + (kk >> 2) * C::QHALF + (kk & 3) * 32, 16, 1024);
              const uint64_t bd = umma_desc_sw128(kb + (kk >> 2) * C::KVHALF + (kk & 3) * 32, 16, 1024);
              umma_ss(sd, ad, bd, C::IDESC_QK, kk > 0 ? 1u : 0u);
            }
            umma_commit(s_full(x, b));
            umma_commit(k_empty + 8 * stage);
          }
          __syncwarp();
        }
      } else {
        const int stage = g % kPxVStages;
        ok = mbar_wait_bounded(v_full + 8 * stage, (g / kPxVStages) & 1);
        const uint32_t vb = sbase + C::V_OFF + stage * C::KBYTES;
        for (int x = 0; x < NT && ok; ++x) {
          ok = __all_sync(0xffffffffu, mbar_wait_bounded(p_full(x, g & 1), (g >> 1) & 1));
          if (!ok) break;
          tc_fence_after();
          const uint32_t pt = tmem + x * 256 + (g & 1) * kPxBN;
          const uint32_t od = tmem + x * 256 + 128;
          if (elect_one()) {
#pragma unroll
            for (int k16 = 0; k16 < kPxBN / 16; ++k16)
              umma_ts(od, pt + k16 * 8, umma_desc_sw128(vb + k16 * 2048, C::KVHALF, 1024),
                      C::IDESC_PV, (!first || k16 > 0) ? 1u : 0u);
            umma_commit(o_done(x));
            umma_commit(p_free(x, g & 1));
            if (x == NT - 1) umma_commit(v_empty + 8 * stage);
          }
          __syncwarp();
        }
      }
      kt = kt + 1 == nkt ? 0 : kt + 1;
    }
    if (!ok && lane == 0) record_error(PKV_DEVERR_TIMEOUT);
    if (elect_one()) umma_commit(mma_idle);
    __syncwarp();
    mbar_wait_bounded(mma_idle, 0);
  } else if ((warp >> 2) < NT) {
    // =================== softmax warps: warps 0-3 tile A, 4-7 tile B ===================
    const int x = warp >> 2;
    const int row = (warp & 3) * 32 + lane;      // TMEM lane = query row of tile x
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t scol = x * 256, ocol = x * 256 + 128;
    const float sl = p.scale_log2;
    bool ok = true;
    int g = 0;
    long long at = g0;
    while (g < ng && ok) {
      // ---- one segment: steps kt0 .. kt1 - 1 of an item
      const int item = (int)(at / nkt), kt0 = (int)(at - (long long)item * nkt);
      const int kt1 = min(nkt, kt0 + ng - g);
      const int j = item / npairs, pair = item - j * npairs;
      const int r = (pair * NT + x) * kT5Rows + row;
      bool valid = r < R;
      const int t = valid ? r / p.G : 0;
      const int h = j * p.G + (valid ? r - t * p.G : 0);
      int last = P - 1;                          // last prefix key this row sees
      if (valid) {
        int s, i, n, L;
        valid = px_row(p, t, s, i, n, L);
        if (valid) last = min(last, L - n + i);
      }
      int lw = last;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) lw = min(lw, __shfl_xor_sync(0xffffffffu, lw, o));
      {
        // Q of the segment in front is free: its last S has been read
        const uint4* qrow = reinterpret_cast<const uint4*>(p.q + ((int64_t)t * p.H_q + h) * D);
        uint8_t* qt = smem + C::Q_OFF + x * C::QBYTES;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          const uint4 v = valid ? __ldg(qrow + c) : make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4*>(qt + (c >> 3) * C::QHALF + row * 128 +
                                    (((c & 7) ^ (row & 7)) << 4)) = v;
        }
        fence_proxy_async_smem();
        mbar_arrive(q_full(x));
      }
      float m_used = 0.f, l = 0.f;
      for (int kt = kt0; kt < kt1 && ok; ++kt, ++g) {
        const int b = g & 1;
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(s_full(x, b), (g >> 1) & 1));
        if (!ok) break;
        tc_fence_after();
        float xs[kPxBN];
        tmem_ld64_wait(tmem + lane_base + scol + b * kPxBN, xs);
        const int kbase = kt * kPxBN;
        if (kbase + kPxBN - 1 > lw) {
          const int lim = last - kbase;
#pragma unroll
          for (int e = 0; e < kPxBN; ++e) xs[e] = e <= lim ? xs[e] : -INFINITY;
        }
        // row maximum: four chains of three-input max over the 64 scores
        float m4[4] = {fmax3(xs[0], xs[1], xs[2]), fmax3(xs[3], xs[4], xs[5]),
                       fmax3(xs[6], xs[7], xs[8]), fmax3(xs[9], xs[10], xs[11])};
#pragma unroll
        for (int e = 12; e + 1 < kPxBN; e += 2) m4[(e >> 1) & 3] = fmax3(m4[(e >> 1) & 3], xs[e], xs[e + 1]);
        const float mt = fmax3(m4[0], m4[1], fmaxf(m4[2], m4[3])) * sl;
        if (kt == kt0) {
          m_used = mt == -INFINITY ? 0.f : mt;
        } else {
          const bool need = mt > m_used + kT5Slack;
          if (__any_sync(0xffffffffu, need)) {
            // O in TMEM is rescaled; O += P(g-1) V must have landed first.  S(g)
            // full implies O += P(g-2) V done, so o_done is at most one phase
            // behind and its parity names the phase unambiguously
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(o_done(x), (g - 1) & 1));
            if (!ok) break;
            tc_fence_after();
            const float mn = need ? mt : m_used;
            const float alpha = exp2f(m_used - mn);
            l *= alpha;
            m_used = mn;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(tmem + lane_base + ocol + c * 32, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st32(tmem + lane_base + ocol + c * 32, o);
            }
            tmem_wait_st();
          }
        }
        // p = 2^(s * scale * log2 e - m): the scale and shift as packed fp32x2 FMAs,
        // the row sum as packed adds
        float2 s2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        const float2 sl2 = make_float2(sl, sl), nm2 = make_float2(-m_used, -m_used);
        uint32_t pk[kPxBN / 2];
#pragma unroll
        for (int c = 0; c < kPxBN / 2; ++c) {
          const float2 y = __ffma2_rn(make_float2(xs[2 * c], xs[2 * c + 1]), sl2, nm2);
          const float2 e2 = make_float2(ex2_approx(y.x), ex2_approx(y.y));
          s2[c & 1] = __fadd2_rn(s2[c & 1], e2);
          pk[c] = pack_bf16x2(e2.x, e2.y);
        }
        l += (s2[0].x + s2[0].y) + (s2[1].x + s2[1].y);
        tmem_st32(tmem + lane_base + scol + b * kPxBN, pk);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(p_full(x, b));
      }
      // ---- the segment's partial state
      if (ok) {
        // the last O += P V of the segment
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(p_free(x, (g - 1) & 1), ((g - 1) >> 1) & 1));
        if (ok) {
          tc_fence_after();
          const int64_t pr = ((int64_t)(cta + item) * NT + x) * kT5Rows + row;
          float4* orow = reinterpret_cast<float4*>(p.o + pr * D);
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(tmem + lane_base + ocol + c * 32, o);
            tmem_wait_ld();
            if (valid) {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                orow[c * 8 + e] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                              __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
            }
          }
          if (valid) p.ml[pr] = make_float2(l > 0.f ? m_used : -INFINITY, l);
          tc_fence_before();                     // O is read before the next segment's P V
        }
      }
      at += kt1 - kt0;
    }
    if (!ok) record_error(PKV_DEVERR_TIMEOUT);
  }

  // ---- teardown: every warp, every path
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, C::TMEM_COLS);
}

// ===========================================================================
// Merge of the partial states of a (token, query head) row: its own tokens'
// (slots of meta[t]) and the prefix's (items[item] = {first CTA, CTAs}).  WPR
// warps per row take eight partials at a time, all of them in flight at once;
// a row's time is that of its loads, and with few rows (a small batch over a
// long prefix) several warps share one.
// ===========================================================================
constexpr int kPxMergeWarps = 8;
constexpr int kPxMergeBatch = 8;

template <int D, int WPR>
__global__ void __launch_bounds__(kPxMergeWarps * 32)
prefix_merge_kernel(const __grid_constant__ PxParams p, int tile_rows) {
  constexpr int V = D / 32, RPC = kPxMergeWarps / WPR;
  __shared__ float s_acc[WPR > 1 ? kPxMergeWarps : 1][D];
  __shared__ float s_m[kPxMergeWarps], s_l[kPxMergeWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = warp % WPR;
  const int pair = blockIdx.x * RPC + warp / WPR;
  const int t = pair / p.H_q, h = pair - t * p.H_q;
  pdl_wait_primary();
  pdl_launch_dependents();
  const int tokens = px_tokens(p.cu, p.S, p.T);
  int s, i, n, L;
  // rows of an inconsistent sequence are left as they are (the decode kernel reports it)
  bool live = t < tokens && px_row(p, t, s, i, n, L);
  int own = 0, np = 0, item = 0, first = 0, base = 0;
  const int j = h / p.G, r = t * p.G + h - j * p.G;
  if (live) {
    const int4 mt = p.meta[t];
    if (p.split.prefix_len > 0) {
      const int npairs = (tokens * p.G + tile_rows - 1) / tile_rows;
      item = j * npairs + r / tile_rows;
      const int2 it = p.items[item];
      first = it.x;
      np = it.y;
    }
    own = mt.y;
    base = mt.x;
    live = own >= 0 && base >= 0 && base + (long long)max(own - 1, 0) * p.own_stride < p.own_slots;
    np += own;
  }
  float M = -INFINITY, lsum = 0.f, acc[V] = {};
  if (live) {
    for (int x0 = sub * kPxMergeBatch; x0 < np; x0 += WPR * kPxMergeBatch) {
      auto index = [&](int x) -> int64_t {
        return x < own ? ((int64_t)base + (int64_t)x * p.own_stride) * p.H_q + h
                       : (int64_t)(first + x - own + item) * tile_rows + r % tile_rows;
      };
      const int cnt = min(kPxMergeBatch, np - x0);
      float2 ml = make_float2(-INFINITY, 0.f);
      if (lane < cnt) ml = (x0 + lane < own ? p.own_ml : p.ml)[index(x0 + lane)];
      float v[kPxMergeBatch][V];
#pragma unroll
      for (int x = 0; x < kPxMergeBatch; ++x)
        if (x < cnt) load_f<V>((x0 + x < own ? p.own_o : p.o) + index(x0 + x) * D + lane * V, v[x]);
      const float m2 = fmaxf(M, warp_max(ml.x));
      const float mu = m2 == -INFINITY ? 0.f : m2;          // nothing visible so far: weights 0
      const float w = exp2f(ml.x - mu), a = exp2f(M - mu);
      M = m2;
      lsum = lsum * a + warp_sum(ml.y * w);
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] *= a;
#pragma unroll
      for (int x = 0; x < kPxMergeBatch; ++x) {
        const float wx = __shfl_sync(0xffffffffu, w, x);
        if (x < cnt) {
#pragma unroll
          for (int e = 0; e < V; ++e) acc[e] = fmaf(wx, v[x][e], acc[e]);
        }
      }
    }
  }
  if constexpr (WPR > 1) {
#pragma unroll
    for (int e = 0; e < V; ++e) s_acc[warp][lane * V + e] = acc[e];
    if (lane == 0) {
      s_m[warp] = M;
      s_l[warp] = lsum;
    }
    __syncthreads();
    if (sub != 0 || !live) return;
    float mu = -INFINITY;
#pragma unroll
    for (int x = 0; x < WPR; ++x) mu = fmaxf(mu, s_m[warp + x]);
    if (mu == -INFINITY) mu = 0.f;
    lsum = 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = 0.f;
#pragma unroll
    for (int x = 0; x < WPR; ++x) {
      const float w = exp2f(s_m[warp + x] - mu);
      lsum += s_l[warp + x] * w;
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] = fmaf(w, s_acc[warp + x][lane * V + e], acc[e]);
    }
  }
  if (!live) return;
  const float inv = lsum > 0.f ? 1.f / lsum : 0.f;          // nothing visible: zeros
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + (int64_t)pair * D + lane * V);
  if constexpr (V == 4)
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv),
                                                pack_bf16x2(acc[2] * inv, acc[3] * inv));
  else
    *dst = pack_bf16x2(acc[0] * inv, acc[1] * inv);
}

}  // namespace pkv
