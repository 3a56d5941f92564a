// Forking block tables: the rows of a group (the beams of a request) continue
// rows of the same group; blocks are shared, a partly filled one is copied, and
// blocks that no row lists any more return to the free ring.
//
// Within a group a block stands at the same entry of every row that lists it
// (rows come from one another by forking), so one thread that sees an entry of
// all rows knows the block's whole reference count: no counters in memory, no
// atomics, and an order of the free blocks that does not depend on timing (by
// group, then entry, then row).  Two launches: the first counts what each group
// takes and gives back, the second sums the counts in front of it, so that every
// CTA knows whether the step fits before anything is written.  Bound by the launches
// and their chains: 22 us for 8 groups of 4 rows, 28 us for 61 of 8 (count 9, apply 12, copy
// 9 when each finds a cold cache) where the bytes take 3.
#pragma once

#include "pkv_copy.cuh"

namespace pkv {

constexpr int kForkThreads = 256;
constexpr int kForkMaxRows = 32;             // rows of a group

struct ForkParams {
  const int32_t* parents;      // [R][B]: row of the group that is continued, -1: none
  const int32_t* lens;         // [R B]
  const int32_t* held;
  const int32_t* shared;       // or null
  const int32_t* tables;
  int32_t* tables_out;         // may be tables
  int32_t* ring;
  const int64_t* state;
  int32_t* lens_out;           // may be lens
  int32_t* held_out;           // may be held
  int64_t* state_out;          // may be state
  int64_t* pairs;              // [R B][2]
  int32_t* totals;
  // workspace
  int64_t* w_state;            // {head, tail}
  int4* w_group;               // [R]: blocks taken, live rows, invalid, 0
  int4* w_row;                 // [R B]: parent, tokens, entries, shared entries of the row
  int32_t* w_give;             // [R][chunks]
  int64_t ring_size;
  int R, B, width, chunks, K;
};

// What a group's rows become.
struct ForkGroup {
  int par[kForkMaxRows];       // row continued, -1: none
  int len[kForkMaxRows];       // its tokens
  int held[kForkMaxRows];      // entries of the new row
  int split[kForkMaxRows];     // entry that gets a fresh block, -1: none
  int had[kForkMaxRows];       // entries of the old row
  int keep[kForkMaxRows];      // leading entries of the old row that are never given back
};

// By one warp; lane i is row i.  Returns whether the row is invalid; `take`: it
// needs a fresh block.
__device__ __forceinline__ bool fork_row(const ForkParams& p, int lane, int parent, int len,
                                         int had, int shared, ForkGroup& f, bool& take) {
  bool bad = false;
  take = false;
  const bool in = lane < p.B;
  if (in)
    bad = parent < -1 || parent >= p.B || len < 0 || had < 0 || had > p.width || shared < 0 ||
          (long long)len > (long long)had * p.K;
  const unsigned bads = __ballot_sync(0xffffffffu, bad);
  if (bads) return bad;
  const bool live = in && parent >= 0;
  const int src = live ? parent : 0;
  const int plen = __shfl_sync(0xffffffffu, len, src), phad = __shfl_sync(0xffffffffu, had, src);
  // the first row that continues a parent goes on in its blocks
  const unsigned alike = __match_any_sync(0xffffffffu, live ? parent : -1 - lane);
  const bool first = (alike & ((1u << lane) - 1)) == 0;
  const int full = plen / p.K, need = full + (plen % p.K ? 1 : 0);
  take = live && !first && need > full;
  if (in) {
    f.par[lane] = live ? parent : -1;
    f.len[lane] = live ? plen : 0;
    f.held[lane] = !live ? 0 : (first ? phad : need);
    f.split[lane] = take ? full : -1;
    f.had[lane] = had;
    f.keep[lane] = shared;
  }
  return false;
}

// Old rows whose entry c goes back: a bit a row.  id: the column's entries
// [row][thread].
__device__ __forceinline__ unsigned fork_given(const ForkGroup& f, int B, int c,
                                               const int32_t (*id)[kForkThreads]) {
  const int t = threadIdx.x;
  unsigned valid = 0, kept = 0;
  for (int b = 0; b < B; ++b)
    if (c < f.had[b]) valid |= 1u << b;
  for (int i = 0; i < B; ++i)
    if (f.par[i] >= 0 && c < f.held[i] && c != f.split[i]) kept |= 1u << f.par[i];
  kept &= valid;
  unsigned give = 0;
  for (int b = 0; b < B; ++b) {
    if (!(valid >> b & 1) || c < f.keep[b] || (kept >> b & 1)) continue;
    // listed by a row that stays, or named by a row in front of this one
    const int x = id[b][t];
    bool stays = false;
    for (int o = 0; o < B; ++o)
      stays |= ((kept >> o & 1) || (o < b && (valid >> o & 1))) && id[o][t] == x;
    if (!stays) give |= 1u << b;
  }
  return give;
}

// Sum over the block.
__device__ __forceinline__ int fork_block_sum(int x, int* s_w) {
  x = __reduce_add_sync(0xffffffffu, x);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s_w[threadIdx.x >> 5] = x;
  __syncthreads();
  int sum = 0;
#pragma unroll
  for (int w = 0; w < kForkThreads / 32; ++w) sum += s_w[w];
  return sum;
}

// grid (groups, chunks of kForkThreads entries)
__global__ void __launch_bounds__(kForkThreads)
fork_count_kernel(const __grid_constant__ ForkParams p) {
  extern __shared__ int32_t s_id[];              // [B][kForkThreads]
  __shared__ ForkGroup s_f;
  __shared__ int s_w[kForkThreads / 32];
  __shared__ int s_bad;
  int32_t(*id)[kForkThreads] = reinterpret_cast<int32_t(*)[kForkThreads]>(s_id);
  const int g = blockIdx.x, chunk = blockIdx.y, tid = threadIdx.x;
  pdl_wait_primary();
  pdl_launch_dependents();
  if (tid < 32) {
    const int64_t row = (int64_t)g * p.B + tid;
    int parent = -1, len = 0, had = 0, shared = 0;
    if (tid < p.B) {
      parent = p.parents[row];
      len = p.lens[row];
      had = p.held[row];
      if (p.shared != nullptr) shared = p.shared[row];
    }
    bool take;
    const bool bad = fork_row(p, tid, parent, len, had, shared, s_f, take);
    const unsigned bads = __ballot_sync(0xffffffffu, bad);
    const unsigned takes = __ballot_sync(0xffffffffu, take);
    const unsigned lives = __ballot_sync(0xffffffffu, tid < p.B && parent >= 0);
    if (chunk == 0) {
      if (tid == 0) {
        p.w_group[g] = make_int4(__popc(takes), __popc(lives), bads != 0, 0);
        if (g == 0) {
          p.w_state[0] = p.state[0];
          p.w_state[1] = p.state[1];
        }
      }
      // (the second launch may write lens and held in place: it reads these)
      if (tid < p.B) p.w_row[row] = make_int4(parent, len, had, shared);
    }
    if (tid == 0) s_bad = bads != 0;
  }
  __syncthreads();
  int n = 0;
  const int c = chunk * kForkThreads + tid;
  if (!s_bad && c < p.width) {
    bool any = false;
    for (int b = 0; b < p.B; ++b)
      if (c < s_f.had[b]) {
        id[b][tid] = p.tables[((int64_t)g * p.B + b) * p.width + c];
        any = true;
      }
    if (any) n = __popc(fork_given(s_f, p.B, c, id));
  }
  n = fork_block_sum(n, s_w);
  if (tid == 0) p.w_give[(int64_t)g * p.chunks + chunk] = n;
}

__global__ void __launch_bounds__(kForkThreads)
fork_apply_kernel(const __grid_constant__ ForkParams p) {
  extern __shared__ int32_t s_id[];              // [B][kForkThreads]
  __shared__ ForkGroup s_f;
  __shared__ int s_w[kForkThreads / 32], s_sum[6][kForkThreads / 32];
  __shared__ int s_rank[kForkMaxRows];           // fresh blocks of the group's earlier rows
  int32_t(*id)[kForkThreads] = reinterpret_cast<int32_t(*)[kForkThreads]>(s_id);
  const int g = blockIdx.x, chunk = blockIdx.y, tid = threadIdx.x;
  pdl_wait_primary();
  // ---- what the groups in front take and give, and all of them
  int take0 = 0, take = 0, live = 0, bad = 0, give0 = 0, give = 0;
  const int64_t head = p.w_state[0], tail = p.w_state[1];
  for (int i = tid; i < p.R; i += kForkThreads) {
    const int4 w = p.w_group[i];
    take += w.x;
    if (i < g) take0 += w.x;
    live += w.y;
    bad |= w.z;
  }
  const int64_t here = (int64_t)g * p.chunks + chunk;
  for (int64_t i = tid; i < (int64_t)p.R * p.chunks; i += kForkThreads) {
    const int n = p.w_give[i];
    give += n;
    if (i < here) give0 += n;
  }
  {
    const int part[6] = {take0, take, give0, give, live, bad};
#pragma unroll
    for (int i = 0; i < 6; ++i) {
      const int x = __reduce_add_sync(0xffffffffu, part[i]);
      if ((tid & 31) == 0) s_sum[i][tid >> 5] = x;
    }
    __syncthreads();
    int sum[6] = {0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 6; ++i)
#pragma unroll
      for (int w = 0; w < kForkThreads / 32; ++w) sum[i] += s_sum[i][w];
    take0 = sum[0]; take = sum[1]; give0 = sum[2]; give = sum[3]; live = sum[4]; bad = sum[5];
  }
  int code = 0;
  if (bad || head < 0 || tail < head || tail - head > p.ring_size ||
      tail + give - head > p.ring_size)
    code = 3;
  else if (take > tail - head)
    code = 1;
  if (g == 0 && chunk == 0 && tid == 0) {
    p.totals[0] = code;
    p.totals[1] = live;
    p.totals[2] = take;
    p.totals[3] = give;
    p.state_out[0] = head + (code ? 0 : take);
    p.state_out[1] = tail + (code ? 0 : give);
    if (code == 3) record_error(PKV_DEVERR_STEP);
  }
  const int c = chunk * kForkThreads + tid;
  const int64_t row0 = (int64_t)g * p.B;
  if (code) {
    // everything as it was
    for (int b = 0; b < p.B; ++b) {
      const int4 w = p.w_row[row0 + b];
      const int64_t at = (row0 + b) * p.width + c;
      if (p.tables_out != p.tables && c < min(w.z, p.width)) p.tables_out[at] = p.tables[at];
      if (chunk == 0 && tid == 0) {
        p.lens_out[row0 + b] = w.y;
        p.held_out[row0 + b] = w.z;
        p.pairs[2 * (row0 + b)] = -1;
        p.pairs[2 * (row0 + b) + 1] = -1;
      }
    }
    return;
  }
  if (tid < 32) {
    int4 w = make_int4(-1, 0, 0, 0);
    if (tid < p.B) w = p.w_row[row0 + tid];
    bool t;
    fork_row(p, tid, w.x, w.y, w.z, w.w, s_f, t);
    const unsigned takes = __ballot_sync(0xffffffffu, t);
    s_rank[tid] = __popc(takes & ((1u << tid) - 1));
    if (chunk == 0 && tid < p.B) {
      p.lens_out[row0 + tid] = s_f.len[tid];
      p.held_out[row0 + tid] = s_f.held[tid];
      if (!t) {
        p.pairs[2 * (row0 + tid)] = -1;
        p.pairs[2 * (row0 + tid) + 1] = -1;
      }
    }
  }
  __syncthreads();
  unsigned back = 0;
  if (c < p.width) {
    bool any = false;
    for (int b = 0; b < p.B; ++b)
      if (c < s_f.had[b]) {
        id[b][tid] = p.tables[(row0 + b) * p.width + c];
        any = true;
      }
    if (any) {
      back = fork_given(s_f, p.B, c, id);
      for (int i = 0; i < p.B; ++i) {
        if (c >= s_f.held[i]) continue;
        const int old = id[s_f.par[i]][tid];
        int x = old;
        if (c == s_f.split[i]) {
          x = p.ring[(head + take0 + s_rank[i]) % p.ring_size];
          p.pairs[2 * (row0 + i)] = old;
          p.pairs[2 * (row0 + i) + 1] = x;
        }
        // (in place most entries stay: beams share their history)
        if (p.tables_out != p.tables || c >= s_f.had[i] || id[i][tid] != x)
          p.tables_out[(row0 + i) * p.width + c] = x;
      }
    }
  }
  // ---- blocks given back: places by entry, then row
  const int n = __popc(back);
  int incl = n;
  const int lane = tid & 31, warp = tid >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  __syncthreads();
  if (lane == 31) s_w[warp] = incl;
  __syncthreads();
  int64_t at = tail + give0 + incl - n;
  for (int w = 0; w < warp; ++w) at += s_w[w];
  while (back) {
    const int b = __ffs(back) - 1;
    back &= back - 1;
    p.ring[at++ % p.ring_size] = id[b][tid];
  }
  // later kernels read tables and lengths before they wait for the kernel in
  // front of them: no early trigger here
  __threadfence();
}

// The tokens of forked rows' partly filled blocks: lens[i] % K leading token
// rows of block pairs[i][0] to block pairs[i][1], K and V, every layer.  grid
// (rows, slices, 2 x layers); a block's leading tokens are contiguous bytes.
struct ForkCopyParams {
  const int64_t* pairs;
  const int32_t* lens;
  uint8_t* k;
  uint8_t* v;
  int64_t k_layer, v_layer;          // bytes of a layer's pool
  int64_t k_row, v_row;              // bytes of a token
  // 4-bit pools: words [layer][block][H][K]; INT8: one word a token (H = 1)
  uint32_t* k_words;
  uint32_t* v_words;
  int64_t num_blocks;
  int K, words;                      // words a token (0: none)
};

constexpr int kForkCopyThreads = 128;
constexpr int kForkCopyUnroll = 4;

template <int VW>
__global__ void __launch_bounds__(kForkCopyThreads)
fork_copy_kernel(const __grid_constant__ ForkCopyParams p) {
  using V = typename VecT<VW>::T;
  pdl_wait_primary();
  pdl_launch_dependents();
  const int64_t i = blockIdx.x;
  const int64_t src = p.pairs[2 * i], dst = p.pairs[2 * i + 1];
  if (src == -1 && dst == -1) return;              // no copy for this row
  const int z = blockIdx.z & 1, layer = blockIdx.z >> 1;
  if (src < 0 || src >= p.num_blocks || dst < 0 || dst >= p.num_blocks) {
    if (threadIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) record_error(PKV_DEVERR_COPY_PAIR);
    return;
  }
  const int len = p.lens[i];
  const int tokens = len > 0 ? len % p.K : 0;
  const int64_t row = z ? p.v_row : p.k_row;
  uint8_t* pool = z ? p.v + layer * p.v_layer : p.k + layer * p.k_layer;
  const V* s = reinterpret_cast<const V*>(pool + src * p.K * row);
  V* d = reinterpret_cast<V*>(pool + dst * p.K * row);
  const int64_t nvec = tokens * row / VW;
  const int64_t first = (int64_t)blockIdx.y * (kForkCopyThreads * kForkCopyUnroll) + threadIdx.x;
  V buf[kForkCopyUnroll];
#pragma unroll
  for (int u = 0; u < kForkCopyUnroll; ++u)
    if (first + u * kForkCopyThreads < nvec) buf[u] = s[first + u * kForkCopyThreads];
#pragma unroll
  for (int u = 0; u < kForkCopyUnroll; ++u)
    if (first + u * kForkCopyThreads < nvec) d[first + u * kForkCopyThreads] = buf[u];
  if (blockIdx.y == 0 && p.words > 0) {
    uint32_t* w = (z ? p.v_words : p.k_words) + layer * p.num_blocks * p.words * p.K;
    for (int e = threadIdx.x; e < p.words * tokens; e += kForkCopyThreads) {
      const int h = e / tokens, t = e - h * tokens;
      w[(dst * p.words + h) * p.K + t] = w[(src * p.words + h) * p.K + t];
    }
  }
}

}  // namespace pkv
