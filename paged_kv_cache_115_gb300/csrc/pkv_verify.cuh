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
// Bound by HBM: one row of p, and one of q where a draft was refused.
#pragma once

#include <cooperative_groups.h>

#include "pkv_copy.cuh"

namespace pkv {

constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyMaxCluster = 16;

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

template <typename T, int E>
struct alignas(sizeof(T) * E) VerifyVec {
  T v[E];
};

template <typename T, int E>
__device__ __forceinline__ void verify_load(const T* row, int x, int V, float (&v)[E]) {
  if (x + E <= V) {
    const VerifyVec<T, E> r = *reinterpret_cast<const VerifyVec<T, E>*>(row + x);
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = to_f32(r.v[e]);
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = x + e < V ? to_f32(row[x + e]) : 0.f;
  }
}

// E: values per vector load (rows and strides are aligned to it).
template <typename T, int E>
__global__ void __launch_bounds__(kVerifyThreads)
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

  // ---- sums of this warp's segment, from p - q, and from p alone where
  // nothing of that is left (a second pass, the same for the whole cluster)
  const int step = 32 * E;
  const int seg = ((V + C * kVerifyWarps - 1) / (C * kVerifyWarps) + step - 1) / step * step;
  const long long lo64 = (long long)(rank * kVerifyWarps + warp) * seg;
  const int lo = (int)min(lo64, (long long)V), hi = (int)min(lo64 + seg, (long long)V);
  bool minus = refused;
  auto weights = [&](int x, float (&w)[E]) {
    verify_load<T, E>(prow, x, V, w);
    if (!minus) return;
    if (qrow != nullptr) {
      float q[E];
      verify_load<T, E>(qrow, x, V, q);
#pragma unroll
      for (int e = 0; e < E; ++e) w[e] -= q[e];
    }
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (x + e == without) w[e] = 0.f;
  };
  // sum of the weights of tiles [a, b) of this warp
  auto sum_of = [&](int a, int b) -> long long {
    long long sum = 0;
    int x = a + lane * E;
    while (x < b) {
      // at most 2048 values to a 32-bit sum of halves below 2^20 + 1
      const int stop = (int)min((long long)b, x + (long long)(2048 / E) * step);
      uint32_t h = 0, l = 0, n = 0;
#pragma unroll 4
      for (; x < stop; x += step) {
        float w[E];
        weights(x, w);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          uint32_t wh, wl;
          verify_halves(w[e], wh, wl);
          h += wh;
          l += wl;
        }
        n += E;
      }
      sum += ((long long)(h - n * kVerifyBias) << 20) + (l - n * kVerifyBias);
    }
    return warp_sum_ll(sum);
  };
  long long total, before;
  for (;;) {
    const long long sum = sum_of(lo, hi);
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
      const int from = (rank * kVerifyWarps + w) * seg, to = min(from + seg, V);
      const int part = ((to - from + kVerifyWarps - 1) / kVerifyWarps + step - 1) / step * step;
      const int pa = min(from + warp * part, to), pb = min(pa + part, to);
      const long long psum = sum_of(pa, pb);
      if (lane == 0) s_part[warp] = psum;
      __syncthreads();
      for (int x = 0; x < warp; ++x) run += s_part[x];
      if (r >= run && r < run + psum) {
        for (int base = pa; base < pb; base += step) {
          const int x = base + lane * E;
          float wt[E];
#pragma unroll
          for (int e = 0; e < E; ++e) wt[e] = 0.f;
          if (x < pb) weights(x, wt);
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
              int found = x;
#pragma unroll
              for (int e = 0; e < E; ++e) {
                if (at <= r) found = x + e;
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
