// Block tables, positions and token slots of one engine step, made from the
// requests' lengths; integer arithmetic throughout.
//
// For request s with lens[s] cached tokens, n new ones (counts[s], -1: over)
// and held[s] listed blocks:
//   ctx = lens + n (0 when over), need = ceil(ctx / K),
//   take = max(0, need - held), give = max(0, held - shared) when over,
//   cu[s] / cb[s] = sums of n / take over the requests before s.
// Table entries held .. need - 1 of s become the free blocks head + cb[s] ..
// of the ring, the blocks of a finished request go to the ring's tail.  lens
// <= held * K, so every fresh block starts with a new token: the token at an
// offset 0 writes the table entry, and every token of the block reads its id
// from the ring.  The part of the ring that is taken from and the part that
// is given to never overlap (checked: tail + given - head <= ring size).
#pragma once

#include "pkv_device.cuh"

namespace pkv {

constexpr int kStepThreads = 1024;
constexpr int kStepFusedTokens = 4096;   // up to here the one CTA does the token rows too

struct StepParams {
  const int32_t* lens;
  const int32_t* counts;
  int32_t* tables;
  const int32_t* held;
  const int32_t* shared;      // may be null
  int32_t* ring;
  const int64_t* state;       // {head, tail}
  int32_t* ctx;               // may be lens
  int32_t* cu;
  int32_t* cb;
  int32_t* positions;
  int64_t* slots;
  int32_t* held_out;          // may be held
  int64_t* state_out;         // may be state
  int32_t* totals;
  int64_t ring_size;
  int64_t num_blocks;
  int max_blocks;
  int S;
  int T;                      // rows of positions / slots
  int K;
  int log2_k;                 // >= 0: K is a power of two
  int wide;                   // positions and slots are 16-byte aligned
};

struct StepRequest {
  long long n;                // new tokens
  int take, give, first;      // blocks taken, given back, first entry given back
  int ctx, held;
  bool bad;
};

__device__ __forceinline__ StepRequest step_request(const StepParams& p, int s) {
  StepRequest r{};
  if (s >= p.S) return r;
  const int len = p.lens[s], cnt = p.counts[s], held = p.held[s];
  const int sh = p.shared != nullptr ? p.shared[s] : 0;
  r.held = held;
  r.first = sh;
  const long long cap = (long long)p.max_blocks * p.K;
  const long long ctx = (long long)len + max(cnt, 0);
  r.bad = len < 0 || cnt < -1 || held < 0 || held > p.max_blocks || sh < 0 ||
          len > (long long)held * p.K || ctx > cap;
  if (r.bad) return r;
  if (cnt < 0) {
    r.give = max(0, held - sh);
    return r;
  }
  r.n = cnt;
  r.ctx = (int)ctx;
  r.take = max(0, (int)((ctx + p.K - 1) / p.K) - held);
  return r;
}

// Exclusive sums of (n; take and give packed in one 64-bit word, both below
// 2^31) over the block; totals returned through tn / tp.  s_a, s_b: 32 words.
__device__ __forceinline__ void step_scan(long long& n, long long& pk, long long& tn,
                                          long long& tp, long long* s_a, long long* s_b) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long n0 = n, p0 = pk;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, n, o), b = __shfl_up_sync(0xffffffffu, pk, o);
    if (lane >= o) {
      n += a;
      pk += b;
    }
  }
  __syncthreads();
  if (lane == 31) {
    s_a[warp] = n;
    s_b[warp] = pk;
  }
  __syncthreads();
  if (warp == 0) {
    long long a = s_a[lane], b = s_b[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
      if (lane >= o) {
        a += x;
        b += y;
      }
    }
    s_a[lane] = a;
    s_b[lane] = b;
  }
  __syncthreads();
  n += (warp ? s_a[warp - 1] : 0) - n0;
  pk += (warp ? s_b[warp - 1] : 0) - p0;
  tn = s_a[31];
  tp = s_b[31];
}

// What the token rows need of their requests, in global memory (the outputs
// of the call) or, for a small step, in shared memory.
struct StepView {
  const int32_t* cu;
  const int32_t* cb;
  const int32_t* ctx;
  const int32_t* held_out;
  int total;                // tokens of the step
  int64_t head;             // head of the ring, modulo its size
};

// The request that holds token t, among requests lo .. hi - 1 (cu[lo] <= t < cu[hi]).
__device__ __forceinline__ int step_find(const int32_t* cu, int lo, int hi, int t) {
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

// Position and slot of token t of request s: from an old table entry or a
// fresh block of the ring, whose first token writes the entry.
__device__ __forceinline__ void step_token(const StepParams& p, const StepView& v, int s, int t,
                                           int& pos, int64_t& slot) {
  const int b0 = v.cb[s], take = v.cb[s + 1] - b0;
  pos = v.ctx[s] - (v.cu[s + 1] - t);
  const int held = v.held_out[s] - take;
  const int lb = p.log2_k >= 0 ? pos >> p.log2_k : pos / p.K;
  const int off = pos - lb * p.K;
  int32_t* entry = p.tables + (int64_t)s * p.max_blocks + lb;
  int id;
  if (lb < held) {
    id = *entry;
  } else {
    int64_t at = v.head + b0 + (lb - held);       // below twice the ring
    if (at >= p.ring_size) at -= p.ring_size;
    id = p.ring[at];
    if (off == 0) *entry = id;
  }
  slot = -1;
  if (id < 0 || id >= p.num_blocks)
    record_error(PKV_DEVERR_BLOCK_ID);
  else
    slot = (int64_t)id * p.K + off;
}

// One CTA: checks, sums, per-request outputs and the blocks given back.
// WITH_TOKENS: the token rows too.
template <bool WITH_TOKENS>
__global__ void __launch_bounds__(kStepThreads)
step_requests_kernel(const __grid_constant__ StepParams p) {
  __shared__ long long s_a[32], s_b[32];
  __shared__ int s_bad;
  // small steps: the token rows find their requests in shared memory
  __shared__ int32_t s_cu[WITH_TOKENS ? kStepThreads + 1 : 1], s_cb[WITH_TOKENS ? kStepThreads + 1 : 1];
  __shared__ int32_t s_ctx[WITH_TOKENS ? kStepThreads : 1], s_held[WITH_TOKENS ? kStepThreads : 1];
  const int tid = threadIdx.x, lane = tid & 31;
  const bool local = WITH_TOKENS && p.S <= kStepThreads;
  pdl_wait_primary();
  // without the token rows the next kernel is step_tokens_kernel, which waits
  // for this one before it reads anything
  if (!WITH_TOKENS) pdl_launch_dependents();
  const int64_t head = p.state[0], tail = p.state[1];
  if (tid == 0) s_bad = 0;
  __syncthreads();
  // ---- what the step asks for
  long long n = 0, pk = 0;
  bool bad = false;
  for (int s = tid; s < p.S; s += kStepThreads) {
    const StepRequest r = step_request(p, s);
    n += r.n;
    pk += (long long)r.take << 32 | (unsigned)r.give;
    bad |= r.bad;
  }
  if (bad) s_bad = 1;
  long long tn, tp;
  step_scan(n, pk, tn, tp, s_a, s_b);
  const long long take = tp >> 32, give = tp & 0xffffffffLL;
  int code = 0;
  if (s_bad || head < 0 || tail < head || tail - head > p.ring_size ||
      tail + give - head > p.ring_size)
    code = 3;
  else if (tn > p.T)
    code = 2;
  else if (take > tail - head)
    code = 1;
  __syncthreads();
  if (tid == 0) {
    p.totals[0] = code;
    p.totals[1] = (int)min(tn, (long long)INT32_MAX);
    p.totals[2] = (int)take;
    p.totals[3] = (int)give;
    p.state_out[0] = head + (code ? 0 : take);
    p.state_out[1] = tail + (code ? 0 : give);
    p.cu[0] = 0;
    p.cb[0] = 0;
    s_cu[0] = s_cb[0] = 0;
    if (code >= 2) record_error(PKV_DEVERR_STEP);
  }
  // ---- per request
  long long cn = 0, cp = 0;             // sums of the earlier tiles
  for (int s0 = 0; s0 < p.S; s0 += kStepThreads) {
    const int s = s0 + tid;
    if (code) {
      if (s < p.S) {
        p.ctx[s] = p.lens[s];
        p.held_out[s] = p.held[s];
        p.cu[s + 1] = 0;
        p.cb[s + 1] = 0;
      }
      continue;
    }
    const StepRequest r = step_request(p, s);
    long long en = r.n, ep = (long long)r.take << 32 | (unsigned)r.give;
    step_scan(en, ep, tn, tp, s_a, s_b);
    en += cn;
    ep += cp;
    if (s < p.S) {
      const bool over = p.counts[s] < 0;
      p.ctx[s] = r.ctx;
      p.held_out[s] = over ? 0 : r.held + r.take;
      p.cu[s + 1] = (int)(en + r.n);
      p.cb[s + 1] = (int)(ep >> 32) + r.take;
      if (local) {
        s_ctx[s] = r.ctx;
        s_held[s] = over ? 0 : r.held + r.take;
        s_cu[s + 1] = (int)(en + r.n);
        s_cb[s + 1] = (int)(ep >> 32) + r.take;
      }
    }
    // a warp gives back the blocks of its 32 requests, one after the other
    unsigned todo = __ballot_sync(0xffffffffu, r.give > 0);
    while (todo) {
      const int l = __ffs(todo) - 1;
      todo &= todo - 1;
      const int give_l = __shfl_sync(0xffffffffu, r.give, l);
      const int first = __shfl_sync(0xffffffffu, r.first, l);
      const int64_t to = tail + __shfl_sync(0xffffffffu, (int)(ep & 0xffffffffLL), l);
      const int32_t* row = p.tables + (int64_t)(s - lane + l) * p.max_blocks + first;
      int64_t at = to % p.ring_size + lane;
      for (int i = lane; i < give_l; i += 128) {          // four loads in flight
        int32_t id[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (i + 32 * u < give_l) id[u] = row[i + 32 * u];
#pragma unroll
        for (int u = 0; u < 4; ++u, at += 32) {
          if (at >= p.ring_size) at -= p.ring_size;
          if (i + 32 * u < give_l) p.ring[at] = id[u];
        }
      }
    }
    cn += tn;
    cp += tp;
  }
  if constexpr (WITH_TOKENS) {
    __syncthreads();
    StepView v = {p.cu, p.cb, p.ctx, p.held_out, code ? 0 : (int)cn, head % p.ring_size};
    if (local) v = {s_cu, s_cb, s_ctx, s_held, v.total, v.head};
    for (int t = tid; t < p.T; t += kStepThreads) {
      int pos = -1;
      int64_t slot = -1;
      if (t < v.total) step_token(p, v, step_find(v.cu, 0, p.S, t), t, pos, slot);
      p.positions[t] = pos;
      p.slots[t] = slot;
    }
  }
  // later kernels read the tables and lengths before they wait for the
  // kernel in front of them: no early trigger here, and everything is
  // visible before the block ends
  __threadfence();
}

// Token rows of a large step: a warp takes 128 of them, four consecutive ones
// a lane, and looks for the requests of its first and last row with 32 probes
// at a time.  Its own bound are the 12 bytes written per row: 1.9 us for 1.06
// million of them.  Both launches take 14.3 us for these rows of 509 requests,
// most of it the one CTA in front (a row a thread with a search each: 19.4).
constexpr int kStepTokenThreads = 256;
constexpr int kStepTokenRows = 4 * kStepTokenThreads;

__device__ __forceinline__ int step_find_warp(const int32_t* cu, int n, int t, int lane) {
  int lo = 0, hi = n;                               // cu[lo] <= t < cu[hi]
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) >> 5, at = lo + lane * step;
    const unsigned le = __ballot_sync(0xffffffffu, at < hi && cu[at] <= t);
    lo += (31 - __clz(le)) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

__global__ void __launch_bounds__(kStepTokenThreads)
step_tokens_kernel(const __grid_constant__ StepParams p) {
  const int lane = threadIdx.x & 31;
  const int w0 = blockIdx.x * kStepTokenRows + (threadIdx.x >> 5) * 128;
  pdl_wait_primary();
  StepView v = {p.cu, p.cb, p.ctx, p.held_out, p.cu[p.S], 0};
  int pos[4];
  int64_t slot[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) pos[u] = -1, slot[u] = -1;
  const int t0 = w0 + 4 * lane;
  if (w0 < v.total) {
    v.head = (p.state_out[0] - p.totals[2]) % p.ring_size;
    const int first = step_find_warp(v.cu, p.S, w0, lane);
    const int last = step_find_warp(v.cu, p.S, min(w0 + 127, v.total - 1), lane);
    if (t0 < v.total) {
      int s = step_find(v.cu, first, last + 1, t0);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int t = t0 + u;
        if (t < v.total) {
          while (t >= v.cu[s + 1]) ++s;
          step_token(p, v, s, t, pos[u], slot[u]);
        }
      }
    }
  }
  // (16-byte stores where the rows' ends and the arrays allow them)
  if (t0 <= p.T - 4 && p.wide) {
    *reinterpret_cast<int4*>(p.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    *reinterpret_cast<longlong2*>(p.slots + t0) = make_longlong2(slot[0], slot[1]);
    *reinterpret_cast<longlong2*>(p.slots + t0 + 2) = make_longlong2(slot[2], slot[3]);
  } else {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (t0 + u < p.T) {
        p.positions[t0 + u] = pos[u];
        p.slots[t0 + u] = slot[u];
      }
    }
  }
  __threadfence();
}

}  // namespace pkv
