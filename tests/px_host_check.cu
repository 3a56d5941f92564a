// Host check of how the prefix kernel's work is cut (pkv_prefix.cuh): every
// step of every item belongs to exactly one CTA, every CTA has one, the item
// table names the CTAs that hold an item's steps, partial slots are distinct
// and inside the workspace, and both kernels' shares of the SMs add up.
#include <cstdio>
#include <cstdlib>
#include <random>
#include <set>
#include <vector>

#include "pkv_prefix.cuh"

#define CHECK(c)                                                             \
  do {                                                                       \
    if (!(c)) {                                                              \
      printf("line %d: %s (heads %d nkt %d ntiles %d n1 %d)\n", __LINE__, #c, heads, nkt, ntiles, n1); \
      return 1;                                                              \
    }                                                                        \
  } while (0)

int main() {
  std::mt19937 rng(5);
  auto pick = [&](int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); };
  int even = 0;
  for (int round = 0; round < 20000; ++round) {
    const int heads = pick(1, 9), nkt = round % 3 ? pick(1, 12) : pick(1, 300);
    const int ntiles = pick(1, 7), npairs = (ntiles + 1) / 2;
    pkv::PxSplit x = {};
    x.prefix_len = nkt * pkv::kPxKeys - pick(0, pkv::kPxKeys - 1);
    x.groups = pick(1, 3);
    x.sms = pick(x.groups + 1, 152);
    x.w1 = pick(1, 100);
    x.w2 = pick(1, 100);
    x.w3 = pick(0, 200);
    const long long work = (long long)heads * nkt * ntiles;
    const long long chunks = pick(0, 3) ? pick(1, 5000) : 0;
    const int n1 = pkv::px_ctas(x, work, chunks, pick(1, 200));
    const pkv::PxCut cut = pkv::px_cut(n1, heads, nkt, ntiles);
    even += cut.per_head > 0;
    CHECK(pkv::px_key_tiles(x.prefix_len) == nkt);
    CHECK(n1 >= 1 && n1 <= x.sms);
    if (chunks > 0) CHECK(n1 == 1 || n1 <= x.sms - x.groups);
    CHECK(pkv::px_ctas(x, 0, chunks, 3) == 0);
    const long long all = (long long)npairs * heads * nkt;
    std::vector<int> owner(all, -1);
    CHECK(cut.n >= 1 && cut.n <= n1);
    for (int c = 0; c < cut.n; ++c) {
      long long g0, g1;
      pkv::px_cta_steps(cut, c, heads, nkt, ntiles, g0, g1);
      CHECK(g0 < g1 && g0 >= 0 && g1 <= all);
      for (long long g = g0; g < g1; ++g) {
        CHECK(owner[g] == -1);
        owner[g] = c;
      }
    }
    std::set<int> slots;
    for (int item = 0; item < npairs * heads; ++item) {
      const int2 at = pkv::px_item_ctas(cut, item, heads, nkt, ntiles);
      const int a = at.x, b = at.x + at.y - 1;
      CHECK(owner[(long long)item * nkt] == a && owner[(long long)(item + 1) * nkt - 1] == b);
      for (int c = a; c <= b; ++c) {
        CHECK(slots.insert(c + item).second);                // a partial state each
        CHECK(c + item < x.sms + npairs * heads);
        bool holds = false;
        for (int s = 0; s < nkt; ++s) holds = holds || owner[(long long)item * nkt + s] == c;
        CHECK(holds);
      }
    }
  }
  if (even < 1000 || even > 19000) return printf("even %d\n", even), 1;
  printf("prefix work ok\n");
  return 0;
}
