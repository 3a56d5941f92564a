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
// stream-K decode kernel on the tokens from prefix_len on (on all tokens of a
// sequence with a row that does not see the whole prefix: px_first).  The first is bound
// by the tensor cores (or, with one tile of rows, by HBM), the second by HBM;
// they run side by side on disjoint SMs: the prefix kernel releases its
// dependent launch at once, the decode kernel does not wait for it, and both
// derive from the lengths on the device how many of the SMs each takes.  The
// merge waits for both.
#pragma once

#include "pkv_attention_tc.cuh"
#include "pkv_prefill_tc05.cuh"
#include "pkv_reduce.cuh"

namespace pkv {

constexpr int kPxBN = kPxKeys;        // keys per step
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
  static constexpr int QBYTES = 2 * QHALF;                // one query tile (64 fp32 values of O too)
  static constexpr int OROW = 256;
  static constexpr int KVHALF = kPxBN * 128;              // 16 KiB
  static constexpr int KBYTES = NH * KVHALF;              // one K (or V) tile
  static constexpr int NS = D == 128 ? 5 : 8;             // ring of K and V tiles in turn
  static constexpr int Q_OFF = 0;                         // [tile][half]
  static constexpr int KV_OFF = 2 * QBYTES;
  static constexpr int BAR_OFF = KV_OFF + NS * KBYTES;
  // full[NS], empty[NS]; per S buffer: p_free, p_full[2]; per query tile:
  // s_full[2], o_done, q_full; mma_idle
  static constexpr int NBAR = 2 * NS + 2 * 3 + 2 * 4 + 1;
  static constexpr int SLOT_OFF = BAR_OFF + 8 * NBAR;
  static constexpr int SMEM = SLOT_OFF + 16 + 1024;
  // S buffers 0, 1 (128 columns each: fp32 S, then P as bf16 pairs: of the
  // lower 64 keys the lo terms, then the hi terms, then of the upper keys), O
  // of tile A, O of tile B (128 each)
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

// Whether packed token t belongs to a consistent sequence s: cu[s] <= t <
// cu[s+1] <= T and n <= its length.  `whole`: its rows see the whole prefix.
__device__ __forceinline__ bool px_row(const PxParams& p, int t, bool& whole) {
  int s = t, n = 1;
  whole = false;
  if (p.cu != nullptr) {
    int lo = 0, hi = p.S;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.cu[mid] <= t) lo = mid; else hi = mid;
    }
    s = lo;
    const int c0 = p.cu[s], c1 = p.cu[s + 1];
    n = c1 - c0;
    if (t < c0 || t >= c1 || c0 < 0 || c1 > p.T || n > p.split.max_q) return false;
  }
  const int cap = min(p.max_len, p.row_tokens);
  const int L = max(0, min(p.lens[s], cap));
  whole = px_first(p.split.prefix_len, n, L) == p.split.prefix_len;
  return p.cu == nullptr || n <= L;
}

// One lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(p));
  return p != 0;
}

// The 128 softmax threads of a tile wait for one another.
__device__ __forceinline__ void px_tile_sync(int x) {
  asm volatile("bar.sync %0, 128;" ::"r"(1 + x) : "memory");
}

// The same, and whether all of them say so: a warp that gave up on a wait
// still gets here, so that no other one waits for it.
__device__ __forceinline__ bool px_tile_all(int x, bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\tbar.red.and.pred q, %1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"(1 + x), "r"((uint32_t)ok)
      : "memory");
  return all != 0;
}

// 16 consecutive 32-bit columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15,%16};"
      :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]),
        "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]),
        "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
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
// Prefix part.  An item is a KV head and up to two tiles of 128 query rows;
// it takes a step per 128 prefix keys.  A run of one item's steps in CTA c is
// one partial state, in slot c + item (distinct, since the runs go through
// CTAs and items in one order).
//
// A job is one query tile's step: S = Q K^T into one of two S buffers (jobs
// take them in turn), softmax, O += P V.  With two tiles an item the jobs of
// the tiles alternate, so one tile's softmax runs under the other's products,
// which share every K and V tile; with one tile the jobs of consecutive
// steps do.  Warps 0-3: softmax of tile A, 4-7: of tile B (one thread per
// query row = TMEM lane); warp 8: TMA producer of K tiles, warp 10: of V
// tiles; warp 9: TMEM and the S products; warp 11: the O products.
//
// A thread reads S twice: both halves of 64 keys for the row maximum, the
// upper one kept, then the lower one again, so that 64 scores are live at a
// time.  A half's P overwrites its part of the S buffer (read by then), and
// the upper keys' product starts while the lower keys' weights are computed.
// P enters as two bf16 terms, hi + lo (the tensor cores take both operands of
// a product in one type, and V is bf16): a weight is off by less than 2^-14
// of itself, where one bf16 term would be off by up to 2^-8, the same for all
// keys of one weight, as much as the output's own rounding and more where
// values cancel.  The row sum l adds the weights in fp32.
// The exponent base of a row is raised only when its maximum grows by more
// than 2^8, so O is rescaled in TMEM rarely.  Every wait is bounded.
//
// On all SMs: 1024 x 32 rows over 16384 tokens (275 GFLOP, 412 with the lo
// terms' products) 297 us, bound by the tensor cores (two jobs take 5150 cycles
// for 4550 of products; with one term 3600 for 3030, 208 us); 8 x 64 rows over
// 131072 tokens (537 MB) 84.6 us, 6.3 TB/s, bound by HBM (82.5 with one term).
// ===========================================================================

// How the steps of all items are dealt to at most n1 CTAs.
// Even: every CTA takes one run of one item, `duo` CTAs for an item of two
// tiles and `solo` for the last item of an odd number of tiles (per_head of
// them for a KV head), the steps of an item shared evenly.  Else (duo = solo =
// 0) the tile steps are dealt out evenly and a CTA may go from one item to the
// next, which costs it the start and end of a second run; taken when rounding
// to whole CTAs would cost more than six tile steps, and with more items than
// CTAs.  Any bound from 3 to 12 does; with 0 the runs of 8 x 64 rows over
// 131072 tokens cross items (97.5 us against 95.1) and of 61 x ~2.5 x 16 over
// 4112 (40.3 against 38.1), without a bound 512 x 32 rows of head_dim 64 over
// 8192 take 152 us against 119.
struct PxCut {
  int n, duo, solo, per_head;
};
__host__ __device__ __forceinline__ PxCut px_cut(int n1, int heads, int nkt, int ntiles) {
  const int npairs = (ntiles + 1) >> 1, share = n1 / heads;
  const long long work = (long long)heads * nkt * ntiles;
  PxCut c = {n1, 0, 0, 0};
  if (n1 < 1 || share < npairs) return c;
  const int odd = ntiles & 1, full = npairs - odd;
  int duo = full ? 2 * share / ntiles : 0;
  if (full && duo < 1) return c;
  if (duo > nkt) duo = nkt;
  int solo = odd ? share - full * duo : 0;
  if (odd && solo < 1) return c;
  if (solo > nkt) solo = nkt;
  const int a = full ? 2 * ((nkt + duo - 1) / duo) : 0, b = odd ? (nkt + solo - 1) / solo : 0;
  if ((a > b ? a : b) > work / n1 + 6) return c;
  c.duo = duo;
  c.solo = solo;
  c.per_head = full * duo + solo;
  c.n = c.per_head * heads;
  return c;
}

// First step (item * nkt + step) that begins at or behind a tile step.
__host__ __device__ __forceinline__ long long px_step_at(long long unit, int nkt, int ntiles) {
  const int npairs = (ntiles + 1) >> 1;
  const long long head = (long long)nkt * ntiles;
  const int j = (int)(unit / head);
  const long long rem = unit - j * head;
  const int pair = (int)(rem / (2LL * nkt));
  const int nt = 2 * pair + 2 <= ntiles ? 2 : 1;
  const int in = (int)(rem - 2LL * pair * nkt);
  return ((long long)j * npairs + pair) * nkt + (in + nt - 1) / nt;
}
// First tile step of step `step` of an item.
__host__ __device__ __forceinline__ long long px_unit_of(int item, int step, int nkt, int ntiles) {
  const int npairs = (ntiles + 1) >> 1, j = item / npairs, pair = item - j * npairs;
  const int nt = 2 * pair + 2 <= ntiles ? 2 : 1;
  return (long long)j * nkt * ntiles + 2LL * pair * nkt + (long long)step * nt;
}
// Steps [g0, g1) of CTA x (item * nkt + step).
__host__ __device__ __forceinline__ void px_cta_steps(const PxCut& c, int x, int heads, int nkt,
                                                      int ntiles, long long& g0, long long& g1) {
  const int npairs = (ntiles + 1) >> 1;
  if (c.per_head > 0) {
    const int j = x / c.per_head, r = x - j * c.per_head, full = npairs - (ntiles & 1);
    const int pair = c.duo > 0 && r < full * c.duo ? r / c.duo : full;
    const int part = r - pair * c.duo, parts = pair < full ? c.duo : c.solo;
    const long long base = ((long long)j * npairs + pair) * nkt;
    g0 = base + (long long)part * nkt / parts;
    g1 = base + (long long)(part + 1) * nkt / parts;
    return;
  }
  const long long work = (long long)heads * nkt * ntiles;
  g0 = px_step_at(x * work / c.n, nkt, ntiles);
  g1 = x + 1 == c.n ? (long long)npairs * heads * nkt : px_step_at((x + 1) * work / c.n, nkt, ntiles);
}
// {first CTA, CTAs} that hold steps of an item.
__host__ __device__ __forceinline__ int2 px_item_ctas(const PxCut& c, int item, int heads, int nkt,
                                                      int ntiles) {
  if (c.per_head > 0) {
    const int npairs = (ntiles + 1) >> 1, full = npairs - (ntiles & 1);
    const int j = item / npairs, pair = item - j * npairs;
    return make_int2(j * c.per_head + pair * c.duo, pair < full ? c.duo : c.solo);
  }
  const long long work = (long long)heads * nkt * ntiles;
  const int a = cta_of_chunk(px_unit_of(item, 0, nkt, ntiles), work, c.n);
  return make_int2(a, cta_of_chunk(px_unit_of(item, nkt - 1, nkt, ntiles), work, c.n) - a + 1);
}

template <int D>
__global__ void __launch_bounds__(kPxThreads, 1)
prefix_tc05_kernel(const __grid_constant__ PxParams p, int tile_rows) {
  using C = PxCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ long long s_chunks[kPxThreads / 32];
  const uint32_t sbase = smem_u32(smem);
  const uint32_t full = sbase + C::BAR_OFF, empty = full + 8 * C::NS;
  const uint32_t tb0 = empty + 8 * C::NS;
  // s_full belongs to a tile and counts that tile's jobs: the other tile's
  // softmax warps may be several items ahead (past items of one tile), and a
  // parity names a phase only to who has seen every phase before it
  auto s_full = [&](int x, int c) { return tb0 + 16 * x + 8 * (c & 1); };
  auto p_free = [&](int b) { return tb0 + 32 + 8 * b; };
  auto p_full = [&](int b, int half) { return tb0 + 48 + 16 * b + 8 * half; };
  auto o_done = [&](int x) { return tb0 + 80 + 8 * x; };
  auto q_full = [&](int x) { return tb0 + 96 + 8 * x; };
  const uint32_t mma_idle = tb0 + 112;
  uint32_t* slot = reinterpret_cast<uint32_t*>(smem + C::SLOT_OFF);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x;

  // barriers and TMEM while the kernel in front still runs
  if (tid == 0) {
    for (int i = 0; i < C::NS; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(s_full(x, 0), 1);
      mbar_init(s_full(x, 1), 1);
      mbar_init(p_free(x), 1);
      mbar_init(p_full(x, 0), kT5Rows);
      mbar_init(p_full(x, 1), kT5Rows);
      mbar_init(o_done(x), 1);
      mbar_init(q_full(x), kT5Rows);
    }
    mbar_init(mma_idle, 2);
    fence_barrier_init();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(slot), C::TMEM_COLS);
    if (lane == 0) {
      prefetch_tensormap(&p.tmap_k);
      prefetch_tensormap(&p.tmap_v);
    }
  }
  tc_fence_before();
  // ---- the SMs of this part: everything the kernel in front wrote is there
  // after the wait, for the decode kernel too
  pdl_wait_primary();
  pdl_launch_dependents();
  long long chunks = 0;
  bool whole = false;
  for (int s = tid; s < p.S; s += kPxThreads)
    chunks += px_own_chunks(p.split, p.cu, p.T, s,
                            max(0, min(p.lens[s], min(p.max_len, p.row_tokens))), whole);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) chunks += __shfl_xor_sync(0xffffffffu, chunks, o);
  if (lane == 0) s_chunks[warp] = chunks;
  whole = __syncthreads_or(whole);
  tc_fence_after();
  const uint32_t tmem = *slot;
  chunks = 0;
#pragma unroll
  for (int w = 0; w < kPxThreads / 32; ++w) chunks += s_chunks[w];
  const int R = px_tokens(p.cu, p.S, p.T) * p.G;           // query rows per KV head
  const int P = p.split.prefix_len;
  const int ntiles = px_tiles(R), npairs = (ntiles + 1) >> 1;
  const int nkt = px_key_tiles(P);
  const long long work = whole ? (long long)p.H_kv * nkt * ntiles : 0;
  const PxCut cut = px_cut(px_ctas(p.split, work, chunks, p.S), p.H_kv, nkt, ntiles);
  if (cta >= cut.n) {
    if (warp == 9) tmem_dealloc(tmem, C::TMEM_COLS);
    return;
  }
  if (cta == cut.n - 1) {                                  // which CTAs hold steps of each item
    for (int x = tid; x < npairs * p.H_kv; x += kPxThreads)
      p.items[x] = px_item_ctas(cut, x, p.H_kv, nkt, ntiles);
  }
  long long g0, g1;
  px_cta_steps(cut, cta, p.H_kv, nkt, ntiles, g0, g1);
  const int ng = (int)(g1 - g0);                           // steps of this CTA
  const int item0 = (int)(g0 / nkt), kt00 = (int)(g0 - (long long)item0 * nkt);
  // query tiles of an item
  auto tiles_of = [&](int item) -> int { return 2 * (item % npairs) + 2 <= ntiles ? 2 : 1; };

  const int K = p.block_size;

  if (warp == 8 || warp == 10) {
    // =================== TMA producers: warp 8 K tiles, warp 10 V tiles ===================
    // Tile 2 g + kv of the ring.  A lane finds the pool row of a box of 16 (8)
    // rows; one elected lane issues the copies of all of them (16 lanes with a
    // copy each took 74 cycles a copy).
    const int kv = warp == 10;
    const CUtensorMap* map = kv ? &p.tmap_v : &p.tmap_k;
    // the prefix is read once per pair of tiles: kept in L2 when there are several
    const uint64_t policy = npairs > 1 ? l2_policy_evict_normal() : l2_policy_evict_first();
    const bool small = K < 16;                            // 8-token blocks: 8-row boxes
    const int nbox = small ? kPxBN / 8 : kPxBN / 16, box = small ? 8 : 16;
    const int log2_k = (K & (K - 1)) == 0 ? __ffs(K) - 1 : -1;
    auto block_of = [&](int tok) -> int { return log2_k >= 0 ? tok >> log2_k : tok / K; };
    int kt = kt00, item = item0;
    // the table entry of this lane's box, loaded one step ahead
    auto table_entry = [&](int g, int t) -> int {
      const int tok = t * kPxBN + lane * box;
      return lane < nbox && g < ng && tok < P ? p.prefix_table[block_of(tok)] : -1;
    };
    int id_next = table_entry(0, kt);
    int n = kv;
    bool ok = true;
    for (int g = 0; g < ng; ++g, n += 2) {
      const int id = id_next, stage = n % C::NS;
      const int ktn = kt + 1 == nkt ? 0 : kt + 1;
      const int tok = kt * kPxBN + lane * box;
      int row = -32;                                      // past the prefix: zero fill
      if (lane < nbox && tok < P) {
        if (id < 0 || id >= p.num_blocks)
          record_error(PKV_DEVERR_BLOCK_ID);
        else
          row = id * K + (tok - block_of(tok) * K);
      }
      id_next = table_entry(g + 1, ktn);
      const int j = item / npairs;
      ok = __all_sync(0xffffffffu, mbar_wait_bounded(empty + 8 * stage, ((n / C::NS) & 1) ^ 1));
      if (!ok) break;
      int rows[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) rows[i] = __shfl_sync(0xffffffffu, row, i);
      if (elect_one()) {
        const uint32_t dst = sbase + C::KV_OFF + stage * C::KBYTES, bar = full + 8 * stage;
        mbar_arrive_expect_tx(bar, C::KBYTES);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if (i < nbox) {
#pragma unroll
            for (int half = 0; half < C::NH; ++half)
              tma_load_3d(dst + half * C::KVHALF + i * box * 128, map, bar, half * 64, j, rows[i],
                          policy);
          }
        }
      }
      __syncwarp();
      kt = ktn;
      if (kt == 0) ++item;
    }
    if (!ok) {
      if (lane == 0) record_error(PKV_DEVERR_TIMEOUT);
      // do not leave the CTA while our own copies may still land
      for (int i = n - 2; i >= 0 && i >= n - 2 * C::NS; i -= 2)
        mbar_wait_bounded(full + 8 * (i % C::NS), (i / C::NS) & 1);
    }
  } else if (warp == 9 || warp == 11) {
    // =================== MMA issue: warp 9 S = Q K^T, warp 11 O += P V ===================
    // The whole warp walks the loop and one elected lane issues.
    bool ok = true;
    int kt = kt00, item = item0, job = 0, seg[2] = {0, 0}, jobs[2] = {0, 0};
    int nt = tiles_of(item);
    for (int g = 0; g < ng && ok; ++g) {
      const bool first = g == 0 || kt == 0;                // of a segment
      if (first) nt = tiles_of(item);
      const int n = 2 * g + (warp == 11);                  // tile of the ring
      const uint32_t kv = sbase + C::KV_OFF + (n % C::NS) * C::KBYTES;
      if (warp == 9 && first) {
#pragma unroll
        for (int x = 0; x < 2; ++x)
          if (x < nt && ok) ok = mbar_wait_bounded(q_full(x), seg[x]++ & 1);
      }
      ok = __all_sync(0xffffffffu,
                      ok && mbar_wait_bounded(full + 8 * (n % C::NS), (n / C::NS) & 1));
      for (int x = 0; x < nt && ok; ++x, ++job) {
        const int b = job & 1;
        const uint32_t sd = tmem + b * kPxBN;
        if (warp == 9) {
          // S buffer b holds P of job - 2 until its O += P V is done
          ok = __all_sync(0xffffffffu,
                          job < 2 || mbar_wait_bounded(p_free(b), ((job >> 1) - 1) & 1));
          if (!ok) break;
          tc_fence_after();
          const uint32_t qb = sbase + C::Q_OFF + x * C::QBYTES;
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint64_t ad = umma_desc_sw128(qb + (kk >> 2) * C::QHALF + (kk & 3) * 32, 16, 1024);
              const uint64_t bd = umma_desc_sw128(kv + (kk >> 2) * C::KVHALF + (kk & 3) * 32, 16, 1024);
              umma_ss(sd, ad, bd, C::IDESC_QK, kk > 0 ? 1u : 0u);
            }
            umma_commit(s_full(x, jobs[x]));
            if (x == nt - 1) umma_commit(empty + 8 * (n % C::NS));
          }
          __syncwarp();
          ++jobs[x];
        } else {
          const uint32_t od = tmem + 256 + x * 128;
#pragma unroll
          for (int h = 0; h < 2; ++h) {                    // upper keys first
            ok = __all_sync(0xffffffffu, ok && mbar_wait_bounded(p_full(b, h), (job >> 1) & 1));
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int i = 0; i < 8; ++i) {                // hi terms, then lo terms
                const int k4 = i & 3, k16 = (h ? 0 : 4) + k4;
                umma_ts(od, sd + (h ? 0 : 64) + (i < 4 ? 32 : 0) + k4 * 8,
                        umma_desc_sw128(kv + k16 * 2048, C::KVHALF, 1024), C::IDESC_PV,
                        (!first || h > 0 || i > 0) ? 1u : 0u);
              }
              if (h == 1) {
                umma_commit(o_done(x));
                umma_commit(p_free(b));
                if (x == nt - 1) umma_commit(empty + 8 * (n % C::NS));
              }
            }
            __syncwarp();
          }
        }
      }
      kt = kt + 1 == nkt ? 0 : kt + 1;
      if (kt == 0) ++item;
    }
    if (!ok && lane == 0) record_error(PKV_DEVERR_TIMEOUT);
    if (elect_one()) umma_commit(mma_idle);
    __syncwarp();
    mbar_wait_bounded(mma_idle, 0);
  } else if (warp < 8) {
    // =================== softmax warps: warps 0-3 tile A, 4-7 tile B ===================
    const int x = warp >> 2;
    const int row = (warp & 3) * 32 + lane;      // TMEM lane = query row of tile x
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ocol = tmem + lane_base + 256 + x * 128;
    const float sl = p.scale_log2;
    bool ok = true;
    int job0 = 0, done = 0;                      // jobs of earlier segments; jobs of this tile
    int item = item0, kt0 = kt00;
    for (int g = 0; g < ng && ok;) {
      // ---- one segment: steps kt0 .. kt0 + nst - 1 of an item
      const int nst = min(nkt - kt0, ng - g), nt = tiles_of(item);
      if (x < nt) {
        const int j = item / npairs, pair = item - j * npairs;
        const int r = (2 * pair + x) * kT5Rows + row;
        bool valid = r < R;
        const int t = valid ? r / p.G : 0;
        const int h = j * p.G + (valid ? r - t * p.G : 0);
        if (valid) {                             // else zero queries, and a state that nobody reads
          bool sees;
          valid = px_row(p, t, sees) && sees;
        }
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
        for (int st = 0; st < nst; ++st) {
          const int job = job0 + st * nt + x, b = job & 1;
          ok = __all_sync(0xffffffffu, mbar_wait_bounded(s_full(x, done), (done >> 1) & 1));
          if (!ok) break;
          tc_fence_after();
          const uint32_t sd = tmem + lane_base + b * kPxBN;
          const int kbase = (kt0 + st) * kPxBN;
          const bool masked = kbase + kPxBN > P;
          float xs[64];
          // 64 scores from key kbase + 64 h on, those past the prefix (their K
          // and V are zeros) at -inf
          auto load = [&](int h) {
            tmem_ld64_wait(sd + 64 * h, xs);
            if (masked) {
              const int end = P - kbase - 64 * h;
#pragma unroll
              for (int e = 0; e < 64; ++e) xs[e] = e < end ? xs[e] : -INFINITY;
            }
          };
          // row maximum: four chains of three-input max
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            load(h);
#pragma unroll
            for (int e = 0; e < 64; e += 2) m4[(e >> 1) & 3] = fmax3(m4[(e >> 1) & 3], xs[e], xs[e + 1]);
          }
          const float mt = fmax3(m4[0], m4[1], fmaxf(m4[2], m4[3])) * sl;
          if (st == 0) {
            m_used = mt == -INFINITY ? 0.f : mt;
          } else {
            // (no weight yet: every score so far was -inf, and 0 no base)
            const bool none = l == 0.f;
            const bool need = mt > m_used + kT5Slack || (none && mt > -INFINITY);
            if (__any_sync(0xffffffffu, need)) {
              // O in TMEM is rescaled; the O product in front must have landed
              // first (the next one waits for this job's P, so o_done is at
              // most one phase ahead of `done`)
              ok = __all_sync(0xffffffffu, mbar_wait_bounded(o_done(x), (done - 1) & 1));
              if (!ok) break;
              tc_fence_after();
              const float mn = need ? mt : m_used;
              const float alpha = none ? 0.f : exp2f(m_used - mn);
              l *= alpha;
              m_used = mn;
#pragma unroll
              for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tmem_ld32(ocol + c * 32, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                tmem_st32(ocol + c * 32, o);
              }
              tmem_wait_st();
            }
          }
          // p = 2^(s * scale * log2 e - m): the scale and shift as packed fp32x2
          // FMAs, the row sum as packed adds; the upper keys are live already
          float2 s2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          const float2 sl2 = make_float2(sl, sl), nm2 = make_float2(-m_used, -m_used);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (h == 1) load(0);
#pragma unroll
            for (int d = 0; d < 2; ++d) {                  // 32 keys each
              uint32_t hi[16], lo[16];
#pragma unroll
              for (int c = 0; c < 16; ++c) {
                const int e = 32 * d + 2 * c;
                const float2 y = __ffma2_rn(make_float2(xs[e], xs[e + 1]), sl2, nm2);
                const float2 e2 = make_float2(ex2_approx(y.x), ex2_approx(y.y));
                s2[c & 1] = __fadd2_rn(s2[c & 1], e2);
                split_bf16x2_trunc(e2.x, e2.y, hi[c], lo[c]);
              }
              tmem_st16(sd + (h ? 0 : 64) + 32 + 16 * d, hi);
              tmem_st16(sd + (h ? 0 : 64) + 16 * d, lo);
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(p_full(b, h));
          }
          l += (s2[0].x + s2[0].y) + (s2[1].x + s2[1].y);
          ++done;
        }
        // ---- the segment's partial state, after its last O product.  With two
        // tiles the product in front of it is known to be done (this tile's
        // last S waited for it), so o_done's parity names the last one.  With
        // one tile it may be two behind; there p_free of the last job's buffer
        // does (the product two jobs before is done, and any later one on
        // that buffer needs this tile's warps)
        const int job1 = job0 + (nst - 1) * nt + x;
        ok = ok && __all_sync(0xffffffffu,
                              nt == 2 ? mbar_wait_bounded(o_done(x), (done - 1) & 1)
                                      : mbar_wait_bounded(p_free(job1 & 1), (job1 >> 1) & 1));
        ok = px_tile_all(x, ok);
        if (ok) {
          tc_fence_after();
          // rows of O to the workspace, 64 values of all rows at a time through
          // this tile's Q (its last S is done): stored from the lanes, a row
          // each, every 16 bytes would be a transaction of their own
          const int64_t pr0 = (int64_t)(cta + item) * tile_rows + x * kT5Rows;
          uint8_t* qt = smem + C::Q_OFF + x * C::QBYTES;
          const int nrow = min(kT5Rows, R - (2 * pair + x) * kT5Rows);
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            float o[64];
            tmem_ld64_wait(ocol + c * 64, o);
#pragma unroll
            for (int e = 0; e < 16; ++e)
              *reinterpret_cast<float4*>(qt + row * C::OROW + ((e ^ (row & 7)) << 4)) =
                  make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
            px_tile_sync(x);
            for (int i = row; i < nrow * 16; i += kT5Rows) {
              const int rr = i >> 4, e = i & 15;
              *reinterpret_cast<float4*>(p.o + (pr0 + rr) * D + c * 64 + e * 4) =
                  *reinterpret_cast<const float4*>(qt + rr * C::OROW + ((e ^ (rr & 7)) << 4));
            }
            px_tile_sync(x);
          }
          if (valid) p.ml[pr0 + row] = make_float2(l > 0.f ? m_used : -INFINITY, l);
          tc_fence_before();                     // O is read before the next segment's P V
        }
      }
      job0 += nst * nt;
      g += nst;
      kt0 = 0;
      ++item;
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
// (slots of meta[t]) and the prefix's (items[item] = {first CTA, CTAs}).  A
// row costs a chain of loads (length, slots, states), so what counts is how
// many warps are resident and how few instructions each takes.  Many rows of
// few partials (WPR 1): four partials at a time.  A small batch over a long
// prefix has few rows of many partials: WPR warps share a row, eight partials
// each at a time.
// 32768 rows of two to four partials take about 14 us, 512 rows of twenty 4.
// ===========================================================================
constexpr int kPxMergeWarps = 8;

template <int D, int WPR>
__global__ void __launch_bounds__(kPxMergeWarps * 32, WPR == 1 ? 5 : 2)
prefix_merge_kernel(const __grid_constant__ PxParams p, int tile_rows) {
  constexpr int V = D / 32, RPC = kPxMergeWarps / WPR, B = WPR == 1 ? 4 : 8;
  __shared__ float s_acc[WPR > 1 ? kPxMergeWarps : 1][D];
  __shared__ float s_m[kPxMergeWarps], s_l[kPxMergeWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = warp % WPR;
  // a CTA takes RPC heads of one token
  const int per_token = (p.H_q + RPC - 1) / RPC;
  const int t = blockIdx.x / per_token;
  const int h = (blockIdx.x - t * per_token) * RPC + warp / WPR;
  const int j = h / p.G, r = t * p.G + h - j * p.G;
  pdl_wait_primary();
  pdl_launch_dependents();
  const int tokens = px_tokens(p.cu, p.S, p.T);
  bool whole = false;
  // rows of an inconsistent sequence are left as they are (the decode kernel reports it)
  bool live = h < p.H_q && t < tokens && px_row(p, t, whole);
  // partial x < own in slot base + x own_stride of its own tokens, the others
  // in row `at` + (x - own) tile_rows of the prefix slots
  int own = 0, np = 0, at = 0, base = 0;
  if (live) {
    const int4 mt = p.meta[t];
    if (whole && p.split.prefix_len > 0) {
      const int npairs = (px_tiles(tokens * p.G) + 1) >> 1;
      const int item = j * npairs + r / (2 * kT5Rows);
      const int2 it = p.items[item];
      at = (it.x + item) * tile_rows + r % (2 * kT5Rows);
      np = it.y;
    }
    own = mt.y;
    base = mt.x;
    live = own >= 0 && base >= 0 && base + (long long)max(own - 1, 0) * p.own_stride < p.own_slots;
    np += own;
  }
  float M = -INFINITY, lsum = 0.f, acc[V] = {};
  if (live) {
    for (int x0 = sub * B; x0 < np; x0 += WPR * B) {
      // (every lane reads the states of all partials: broadcasts cost less
      // than the shuffles of one state per lane)
      float2 ml[B];
      float v[B][V];
#pragma unroll
      for (int x = 0; x < B; ++x) {
        ml[x] = make_float2(-INFINITY, 0.f);
        if (x0 + x < np) {
          const bool mine = x0 + x < own;
          const int row = mine ? (base + (x0 + x) * p.own_stride) * p.H_q + h
                               : at + (x0 + x - own) * tile_rows;
          ml[x] = (mine ? p.own_ml : p.ml)[row];
          load_f<V>((mine ? p.own_o : p.o) + (int64_t)row * D + lane * V, v[x]);
        }
      }
      float m2 = M;
#pragma unroll
      for (int x = 0; x < B; ++x) m2 = fmaxf(m2, ml[x].x);
      const float mu = m2 == -INFINITY ? 0.f : m2;          // nothing visible so far: weights 0
      const float a = ex2_approx(M - mu);
      M = m2;
      lsum *= a;
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] *= a;
#pragma unroll
      for (int x = 0; x < B; ++x) {
        // (not a partial of which the row sees no key: it may hold 0 x NaN)
        if (ml[x].y != 0.f) {
          const float w = ex2_approx(ml[x].x - mu);
          lsum = fmaf(ml[x].y, w, lsum);
#pragma unroll
          for (int e = 0; e < V; ++e) acc[e] = fmaf(w, v[x][e], acc[e]);
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
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + ((int64_t)t * p.H_q + h) * D + lane * V);
  if constexpr (V == 4)
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv),
                                                pack_bf16x2(acc[2] * inv, acc[3] * inv));
  else
    *dst = pack_bf16x2(acc[0] * inv, acc[1] * inv);
}

}  // namespace pkv
