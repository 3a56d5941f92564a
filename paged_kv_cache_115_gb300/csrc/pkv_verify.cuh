// Verification of drafted tokens: acceptance by given random numbers, and the
// draw of the next token from max(p - q, 0) (or p).
//
// Whole numbers all the way: a weight w counts floor(min(w, 1) 2^40), a sum
// of at most 2^22 of them fits 62 bits, so sums do not depend on their order
// and the drawn token is the same on every machine.  Both factors of u q < p
// have 24 bits, their product is exact in 64-bit floating point.
//
// One cluster of CTAs per sequence.  Each warp sums a contiguous segment of
// the vocabulary; the CTAs exchange their sums through distributed shared
// memory, and the warps of the CTA whose sums hold the threshold share the
// one segment that holds it (read again, from L1 / L2) to find the token.
// Bound by HBM: one row of p, and one of q where a draft was refused, behind
// a chain of about 6 us (counts, tokens, their probabilities, sums, threshold,
// the segment again).  256 sequences over 131072 float32, two in three
// refused: 224 MB in 41.3 us, 5.4 TB/s.  Loops of their own for p, p - q and
// shifted q, eight, four and two tiles in flight, keep two CTAs of 512 threads
// on an SM without spills (one loop for all: 49.7 us).
#pragma once

#include <cooperative_groups.h>

#include "pkv_copy.cuh"

namespace pkv {

constexpr int kVerifyThreads = 512;
constexpr int kVerifyCtas = 2;          // resident on an SM
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyMaxCluster = 8;
constexpr int kVerifyBatch = 4;         // tiles whose loads of p and q are in flight together

struct VerifyParams {
  const void* target;
  const void* draft;            // may be null
  const int32_t* tokens;
  const float* uniforms;
  const int32_t* cu;
  int32_t* out;
  int32_t* num_new;
  int64_t target_stride, draft_seq_stride, draft_tok_stride;
  int num_tokens, max_query, vocab;
};

// floor(min(max(w, 0), 1) 2^40) as (high, low) halves of 20 bits, by two sums
// that truncate: 8 + x keeps floor(x 2^20) in the low mantissa bits (a
// conversion to 64-bit integers runs at a fraction of the rate of these).
// NaN counts 0.  The halves stand above the bits of 8.0f, which callers take
// off once per sum.
constexpr uint32_t kVerifyBias = 0x41000000u;   // bits of 8.0f
__device__ __forceinline__ void verify_halves(float w, uint32_t& hi, uint32_t& lo) {
  w = fminf(fmaxf(w, 0.f), 1.f);
  const float t = __fadd_rz(w, 8.f);
  hi = __float_as_uint(t);
  lo = __float_as_uint(__fmaf_rz(w - (t - 8.f), 1048576.f, 8.f));
}
__device__ __forceinline__ long long verify_weight(float w) {
  uint32_t hi, lo;
  verify_halves(w, hi, lo);
  return ((long long)(hi - kVerifyBias) << 20) + (lo - kVerifyBias);
}

__device__ __forceinline__ long long warp_sum_ll(long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The weights of one sequence's draw, read in 16-byte blocks that are aligned
// on the row of p: block i holds values i E - sp .. of the vocabulary (E = 16
// / sizeof(T); sp values of the first block lie in front of the row).  The row
// of q may sit at another distance from a 16-byte boundary (an odd vocabulary
// does that), so a block of it is cut out of two aligned ones.
template <typename T>
struct VerifyRow {
  static constexpr int E = 16 / sizeof(T);
  static constexpr int TILE = 32 * E;      // values of a tile: one block per lane
  const T* p;
  const T* q;                              // null: nothing comes off
  const uint4* p_al;
  const uint4* q_al;
  int V, sp, without, word, half;          // q's shift: whole words, and 16 bits more
  bool shifted;

  __device__ __forceinline__ VerifyRow(const T* prow, const T* qrow, int vocab, int skip)
      : p(prow), q(qrow), V(vocab), without(skip) {
    const uintptr_t pa = reinterpret_cast<uintptr_t>(prow);
    sp = (int)(pa & 15) / (int)sizeof(T);
    p_al = reinterpret_cast<const uint4*>(pa & ~uintptr_t(15));
    const uintptr_t qa = reinterpret_cast<uintptr_t>(qrow) - (pa & 15);
    const int o = (int)(qa & 15);
    q_al = reinterpret_cast<const uint4*>(qa & ~uintptr_t(15));
    shifted = o != 0;
    word = o >> 2;
    half = (o & 2) * 8;
  }
  __device__ __forceinline__ int tiles() const { return (V + sp + TILE - 1) / TILE; }
  // tiles t .. t + n - 1 lie inside both rows and hold no refused draft
  __device__ __forceinline__ bool inside(int t, int n) const {
    const int a = t * TILE - sp, b = (t + n) * TILE - sp;
    return a >= 0 && b <= V && (without < a || without >= b);
  }
  __device__ __forceinline__ static void unpack(const uint4& r, float (&x)[E]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) {
        x[i] = __uint_as_float(w[i]);
      } else {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    }
  }
  // 16 bytes of (a, b) from byte word * 4 + half / 8 on
  __device__ __forceinline__ uint4 cut(const uint4& a, const uint4& b) const {
    uint32_t v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}, c[5];
#pragma unroll
    for (int i = 0; i < 5; ++i) {
      const uint32_t lo = word & 1 ? v[i + 1] : v[i];
      const uint32_t hi = i + 2 < 8 ? (word & 1 ? (i + 3 < 8 ? v[i + 3] : 0u) : v[i + 2]) : 0u;
      c[i] = word & 2 ? hi : lo;
    }
    return make_uint4(__funnelshift_r(c[0], c[1], half), __funnelshift_r(c[1], c[2], half),
                      __funnelshift_r(c[2], c[3], half), __funnelshift_r(c[3], c[4], half));
  }
  // this lane's block of N tiles that lie inside, all loads first (MODE 0: p,
  // 1: p - q, 2: p - q with q's blocks cut out of two)
  template <int N, int MODE, typename F>
  __device__ __forceinline__ void visit(int t, int lane, F&& f) const {
    uint4 a[N], b[N], c[N];
    const int64_t i0 = (int64_t)t * 32 + lane;
#pragma unroll
    for (int n = 0; n < N; ++n) a[n] = __ldg(p_al + i0 + 32 * n);
    if constexpr (MODE > 0) {
#pragma unroll
      for (int n = 0; n < N; ++n) b[n] = __ldg(q_al + i0 + 32 * n);
    }
    if constexpr (MODE == 2) {
#pragma unroll
      for (int n = 0; n < N; ++n) c[n] = __ldg(q_al + i0 + 32 * n + 1);
#pragma unroll
      for (int n = 0; n < N; ++n) b[n] = cut(b[n], c[n]);
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
      float w[E];
      unpack(a[n], w);
      if constexpr (MODE > 0) {
        float x[E];
        unpack(b[n], x);
#pragma unroll
        for (int e = 0; e < E; ++e) w[e] -= x[e];
      }
      f(w);
    }
  }
  // this lane's block of any tile (0 outside the row)
  __device__ __forceinline__ void block(int t, int lane, float (&w)[E]) const {
    const int x0 = (t * 32 + lane) * E - sp;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int x = x0 + e;
      w[e] = 0.f;
      if (x >= 0 && x < V && x != without) {
        w[e] = to_f32(p[x]);
        if (q != nullptr) w[e] -= to_f32(q[x]);
      }
    }
  }
  template <int MODE>
  __device__ __forceinline__ long long sum_mode(int t0, int t1, int lane) const {
    constexpr int N = MODE == 0 ? 2 * kVerifyBatch : (MODE == 1 ? kVerifyBatch : kVerifyBatch / 2);
    long long total = 0;
    uint32_t h = 0, l = 0, n = 0;
    auto add = [&](const float (&w)[E]) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        uint32_t wh, wl;
        verify_halves(w[e], wh, wl);
        h += wh;
        l += wl;
      }
      n += E;
    };
    for (int t = t0; t < t1;) {
      if (t + N <= t1 && inside(t, N)) {
        visit<N, MODE>(t, lane, add);
        t += N;
      } else if (inside(t, 1)) {
        visit<1, MODE>(t, lane, add);
        ++t;
      } else {
        float w[E];
        block(t, lane, w);
        add(w);
        ++t;
      }
      if (n >= 1024) {         // halves are at most 2^20: 32-bit sums of up to 2048 of them
        total += ((long long)(h - n * kVerifyBias) << 20) + (l - n * kVerifyBias);
        h = l = n = 0;
      }
    }
    total += ((long long)(h - n * kVerifyBias) << 20) + (l - n * kVerifyBias);
    return warp_sum_ll(total);
  }
  // sum of the weights of tiles [t0, t1), of the whole warp
  __device__ __forceinline__ long long sum(int t0, int t1, int lane) const {
    if (q == nullptr) return sum_mode<0>(t0, t1, lane);
    return shifted ? sum_mode<2>(t0, t1, lane) : sum_mode<1>(t0, t1, lane);
  }
};

template <typename T>
__global__ void __launch_bounds__(kVerifyThreads, kVerifyCtas)
verify_kernel(const __grid_constant__ VerifyParams p) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  __shared__ long long s_warp[kVerifyWarps];      // sums of the warps' segments
  __shared__ long long s_part[kVerifyWarps];      // sums of the parts of the threshold's segment
  __shared__ long long s_tot;
  __shared__ int s_accepted, s_bad_draft;
  const int C = cluster.num_blocks(), rank = cluster.block_rank();
  const int s = blockIdx.x / C;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int V = p.vocab;
  pdl_wait_primary();
  pdl_launch_dependents();

  const int c0 = p.cu[s], c1 = p.cu[s + 1], rows = c1 - c0;
  int32_t* out = p.out + (int64_t)s * p.max_query;
  const bool bad = c0 < 0 || rows < 0 || c1 > p.num_tokens || rows > p.max_query;
  if (bad || rows == 0) {               // the same for every CTA of the cluster
    if (rank == 0) {
      if (bad && tid == 0) record_error(PKV_DEVERR_DRAFT);
      for (int i = tid; i < p.max_query; i += kVerifyThreads) out[i] = -1;
      if (tid == 0) p.num_new[s] = 0;
    }
    return;
  }
  const T* target = static_cast<const T*>(p.target);
  const T* draft = static_cast<const T*>(p.draft);
  const int n = rows - 1;
  // ---- accepted drafts
  if (warp == 0) {
    int a = n;
    bool out_of_vocab = false;
    for (int b = 0; b < n; b += 32) {
      const int i = b + lane;
      bool ok = true, oov = false;
      if (i < n) {
        const int d = p.tokens[c0 + 1 + i];
        oov = d < 0 || d >= V;
        ok = false;
        if (!oov) {
          const double pv = to_f32(target[(int64_t)(c0 + i) * p.target_stride + d]);
          const double qv = draft != nullptr
                                ? to_f32(draft[s * p.draft_seq_stride + i * p.draft_tok_stride + d])
                                : 1.f;
          ok = (double)p.uniforms[c0 + i] * qv < pv;
        }
      }
      const unsigned no = __ballot_sync(0xffffffffu, !ok);
      if (no) {
        a = b + __ffs(no) - 1;
        out_of_vocab = __shfl_sync(0xffffffffu, (int)oov, a - b);
        break;
      }
    }
    if (lane == 0) {
      s_accepted = a;
      s_bad_draft = out_of_vocab;
    }
  }
  __syncthreads();
  const int a = s_accepted;
  const bool refused = a < n;
  const T* prow = target + (int64_t)(c0 + a) * p.target_stride;
  // what comes off p: a row of q, or the refused draft alone
  const T* qrow = refused && !s_bad_draft && draft != nullptr
                      ? draft + s * p.draft_seq_stride + a * p.draft_tok_stride : nullptr;
  const int without = refused && !s_bad_draft && draft == nullptr ? p.tokens[c0 + 1 + a] : -1;
  if (rank == 0) {
    for (int i = tid; i < p.max_query; i += kVerifyThreads)
      if (i != a) out[i] = i < a ? p.tokens[c0 + 1 + i] : -1;
    if (tid == 0) {
      p.num_new[s] = a + 1;
      if (refused && s_bad_draft) record_error(PKV_DEVERR_DRAFT);
    }
  }

  // ---- sums of this warp's segment (whole tiles), from p - q, and from p
  // alone where nothing of that is left (a second pass, the same for the
  // whole cluster)
  VerifyRow<T> row(prow, qrow, V, without);
  constexpr int E = VerifyRow<T>::E;
  const int tiles = row.tiles();
  const int seg = (tiles + C * kVerifyWarps - 1) / (C * kVerifyWarps);
  const int lo = min((rank * kVerifyWarps + warp) * seg, tiles), hi = min(lo + seg, tiles);
  bool minus = refused;
  long long total, before;
  for (;;) {
    const long long sum = row.sum(lo, hi, lane);
    if (lane == 0) s_warp[warp] = sum;
    __syncthreads();
    if (warp == 0) {
      const long long w = warp_sum_ll(lane < kVerifyWarps ? s_warp[lane] : 0);
      if (lane == 0) s_tot = w;
    }
    cluster.sync();
    const long long mine = lane < C ? *cluster.map_shared_rank(&s_tot, lane) : 0;
    total = warp_sum_ll(mine);
    before = warp_sum_ll(lane < rank ? mine : 0);
    if (total > 0 || !minus) break;
    minus = false;
    row = VerifyRow<T>(prow, nullptr, V, -1);
    cluster.sync();
  }
  if (total == 0) {
    if (rank == 0 && tid == 0) {
      out[a] = -1;
      record_error(PKV_DEVERR_DRAFT);
    }
  } else {
    const float uf = fminf(fmaxf(p.uniforms[c1 - 1], 0.f), 0.99999994f);
    const long long u = (long long)(uf * 16777216.f);
    const long long r = (total >> 24) * u + (((total & 0xffffffLL) * u) >> 24);
    if (r >= before && r < before + s_tot) {
      // the threshold is in this CTA: its warps share the one segment that
      // holds it, and the warp whose part holds it finds the token
      long long run = before;
      int w = 0;
      while (r >= run + s_warp[w]) run += s_warp[w++];
      const int from = (rank * kVerifyWarps + w) * seg, to = min(from + seg, tiles);
      const int part = (to - from + kVerifyWarps - 1) / kVerifyWarps;
      const int pa = min(from + warp * part, to), pb = min(pa + part, to);
      const long long psum = row.sum(pa, pb, lane);
      if (lane == 0) s_part[warp] = psum;
      __syncthreads();
      for (int x = 0; x < warp; ++x) run += s_part[x];
      if (r >= run && r < run + psum) {
        for (int t = pa; t < pb; ++t) {
          float wt[E];
          row.block(t, lane, wt);
          long long own = 0;
#pragma unroll
          for (int e = 0; e < E; ++e) own += verify_weight(wt[e]);
          long long incl = own;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const long long up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
          }
          const unsigned over = __ballot_sync(0xffffffffu, run + incl > r);
          if (over) {
            if (lane == __ffs(over) - 1) {
              long long at = run + incl - own;
              int found = 0;
#pragma unroll
              for (int e = 0; e < E; ++e) {
                if (at <= r) found = (t * 32 + lane) * E - row.sp + e;
                at += verify_weight(wt[e]);
              }
              out[a] = found;
            }
            break;
          }
          run += __shfl_sync(0xffffffffu, incl, 31);
        }
      }
    }
  }
  cluster.sync();       // no CTA leaves while another reads its sums
}

}  // namespace pkv
