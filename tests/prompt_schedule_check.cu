// Host-only check of how the prompt attention's work is shared out (the same
// __host__ __device__ functions the kernels use).  Prints "ok" and returns 0
// when all of this holds, over ragged batches, grouped heads and grids:
//
//  1. floor_sum_128 and cost_before equal their sums term by term.
//  2. The shares cover every key tile of every item exactly once, in order.
//  3. The pieces of an item are those of consecutive CTAs, the first and the
//     last of which share_owner names, none of them empty.
//  4. A CTA has at most one incomplete item that it began (piece slot 1) and at
//     most one that an earlier CTA began (slot 0).
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "prompt_schedule.cuh"

using namespace qspec;

static int fail(const char* what, long long a, long long b, long long c) {
  std::printf("FAIL %s: %lld %lld %lld\n", what, a, b, c);
  return 1;
}

struct Entry {
  int64_t start;
  int w, n;
};

static unsigned g_state = 12345;
static unsigned rnd(unsigned n) {
  g_state = g_state * 1664525u + 1013904223u;
  return (g_state >> 8) % n;
}

int main() {
  for (int k = 0; k < 40000; ++k) {
    const int64_t n = rnd(k & 1 ? 200 : 20000), b = rnd(k & 2 ? 100000 : 2000000000);
    const int a = k % 3 ? 1 + rnd(256) : 1 << rnd(9);
    int64_t want = 0;
    for (int64_t i = 0; i < n; ++i) want += (a * i + b) / 128;
    if (floor_sum_128(n, a, b) != want) return fail("floor_sum_128", n, a, b);
  }
  const int groups[] = {1, 2, 3, 4, 5, 7, 8, 16, 48, 100, 128};
  const int grids[] = {1, 2, 7, 64, 148};
  long long checked = 0;
  for (int trial = 0; trial < 400; ++trial) {
    const int group = groups[trial % 11], tpt = 128 / group, h_kv = 1 + rnd(4), batch = 1 + rnd(20);
    const int scale = trial % 3 == 0 ? 6 : (trial % 3 == 1 ? 300 : 3000);
    std::vector<Run> runs;
    std::vector<int64_t> starts;
    std::vector<Entry> items;
    int64_t pos = 0;
    auto add = [&](const Run& r) -> int {
      if (r.n == 0) return 0;
      for (int g = 0; g < h_kv; ++g) {
        const int64_t head = pos;
        for (int i = 0; i < run_items(r); ++i) {
          if (head + cost_before(r, i) != pos) return fail("cost_before", r.n, r.base, i);
          const int tokens = item_tokens(r, i);
          if (tokens < 1 || tokens > 2 * r.tpt) return fail("tokens", r.n, i, tokens);
          Entry e;
          e.start = pos;
          e.w = tokens > r.tpt ? 2 : 1;
          e.n = item_tiles(r, i, tokens);
          if (e.n < 1) return fail("tiles", r.n, r.base, i);
          items.push_back(e);
          pos += e.w == 2 ? kTileCost2 * e.n + kItemCost2 : kTileCost1 * e.n + kItemCost1;
        }
        if (run_cost(r) != pos - head) return fail("run_cost", r.n, r.base, g);
      }
      return 0;
    };
    int all = 0;
    for (int b = 0; b < batch; ++b) {
      Run r;
      r.n = rnd(4) == 0 ? 0 : 1 + rnd(scale);
      r.tpt = tpt;
      r.base = rnd(2) ? 0 : rnd(5000);
      r.pre = trial % 5 == 0 ? 1 + trial % 7 : 0;
      all += r.n;
      runs.push_back(r);
    }
    if (trial & 1) {
      Run p;
      p.n = all;
      p.tpt = tpt;
      p.base = -1;
      p.pre = 1 + rnd(70);
      if (add(p)) return 1;
    }
    for (const Run& r : runs)
      if (add(r)) return 1;
    const int64_t total = pos;
    if (total == 0) continue;
    for (int grid : grids) {
      const int ctas = working_ctas(total, grid);
      if (ctas < 1 || ctas > grid) return fail("ctas", total, grid, ctas);
      int64_t reached = 0;
      std::vector<int> next(items.size(), 0), first(items.size(), -1), last(items.size(), -1);
      size_t from = 0;
      for (int c = 0; c < ctas; ++c) {
        int64_t s0, s1;
        share_of(total, ctas, c, &s0, &s1);
        if (s0 != reached || s1 <= s0) return fail("cover", total, ctas, c);
        reached = s1;
        int begun = 0, carried = 0;
        while (from > 0 && items[from].start > s0) --from;
        while (from + 1 < items.size() && items[from + 1].start <= s0) ++from;
        for (size_t i = from; i < items.size() && items[i].start < s1; ++i) {
          int j0, j1;
          share_tiles(items[i].start, items[i].w, items[i].n, s0, s1, &j0, &j1);
          if (j0 >= j1) continue;
          if (j0 != next[i]) return fail("gap", static_cast<long long>(i), j0, next[i]);
          next[i] = j1;
          if (first[i] < 0) first[i] = c;
          else if (last[i] != c - 1) return fail("pieces apart", static_cast<long long>(i), last[i], c);
          last[i] = c;
          if (j0 > 0 || j1 < items[i].n) {
            if (items[i].start < s0) ++carried; else ++begun;
          }
          ++checked;
        }
        if (begun > 1 || carried > 1) return fail("piece slots", c, begun, carried);
      }
      if (reached != total) return fail("cover", total, ctas, reached);
      for (size_t i = 0; i < items.size(); ++i) {
        if (next[i] != items[i].n) return fail("tiles left", static_cast<long long>(i), next[i], items[i].n);
        if (share_owner(total, ctas, items[i].start) != first[i]) return fail("first", static_cast<long long>(i), first[i], ctas);
        if (share_owner(total, ctas, items[i].start + static_cast<int64_t>(items[i].w == 2 ? kTileCost2 : kTileCost1) * (items[i].n - 1)) != last[i])
          return fail("last", static_cast<long long>(i), last[i], ctas);
      }
    }
  }
  std::printf("ok %lld pieces\n", checked);
  return 0;
}
