// How the attention of many tokens (prompt_attention.cuh) is shared out.
//
// A tile is 128 query rows by 128 keys.  The rows of a tile belong to one KV
// head: row r holds query head g * group + r % group of token r / group, so
// grouped heads fill the tile and share its keys.  An item is the work of one
// KV head on a run of at most 2 * tpt tokens (tpt = 128 / group, rounded
// down): two row tiles that share every key tile, or one when tpt tokens or
// fewer are left.  Items, in order:
//   the shared prefix:  for g, for the runs of all packed tokens: prefix_len keys;
//   the sequences:      for b, for g, for the runs of b's tokens: the keys that the run's last token sees.
// An item costs (row tiles) x (key tiles) + kItemCost; the costs of all items
// laid end to end are cut into equal shares, one for each CTA, whatever the
// batch, the lengths and the heads.  A key tile belongs to the CTA in whose
// share its place on that line falls, so a long item is split over CTAs.
// Everything follows from the lengths in closed form (a sum of floors), so
// each CTA finds its share alone.
#pragma once

#include <cstdint>

namespace qspec {

constexpr int kItemCost = 2;       // an item's fixed cost (queries, output) in tiles of 128 x 128
constexpr int kMinShare = 6;       // a CTA's smallest share: fewer CTAs work where there is less

// sum over i < n of floor((a i + b) / m), by Euclid's steps on (a, m).
__host__ __device__ inline int64_t floor_sum(int64_t n, int64_t m, int64_t a, int64_t b) {
  int64_t ans = 0;
  while (n > 0) {
    if (a >= m) {
      ans += (n - 1) * n / 2 * (a / m);
      a %= m;
    }
    if (b >= m) {
      ans += n * (b / m);
      b %= m;
    }
    const int64_t y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y % m;
    const int64_t s = m;
    m = a;
    a = s;
  }
  return ans;
}

// The items of one KV head over a run of n tokens, the first of which sees
// base + 1 keys (causal), or all of which see `keys` (base < 0).
struct Run {
  int n;           // tokens
  int tpt;         // tokens of a row tile
  int64_t base;    // keys before the run's first token; < 0: not causal
  int64_t keys;    // not causal: visible keys
};

__host__ __device__ inline int run_items(const Run& r) { return (r.n + 2 * r.tpt - 1) / (2 * r.tpt); }

__host__ __device__ inline int item_tokens(const Run& r, int i) {
  const int left = r.n - i * 2 * r.tpt;
  return left < 2 * r.tpt ? left : 2 * r.tpt;
}

__host__ __device__ inline int item_row_tiles(const Run& r, int i) { return item_tokens(r, i) > r.tpt ? 2 : 1; }

// Keys that the first `tokens` tokens of item i see at most.
__host__ __device__ inline int64_t item_keys(const Run& r, int i, int tokens) {
  return r.base < 0 ? r.keys : r.base + static_cast<int64_t>(i) * 2 * r.tpt + tokens;
}

__host__ __device__ inline int64_t item_cost(const Run& r, int i) {
  return item_row_tiles(r, i) * ((item_keys(r, i, item_tokens(r, i)) + 127) / 128) + kItemCost;
}

// The cost of the items before item i (i <= run_items(r)).
__host__ __device__ inline int64_t cost_before(const Run& r, int i) {
  int64_t last = 0;
  if (i > 0 && item_tokens(r, i - 1) < 2 * r.tpt) {      // only a run's last item is not full
    last = item_cost(r, i - 1);
    --i;
  }
  const int64_t s = 2 * r.tpt;
  const int64_t tiles = r.base < 0 ? i * ((r.keys + 127) / 128) : floor_sum(i, 128, s, r.base + s + 127);
  return 2 * tiles + static_cast<int64_t>(i) * kItemCost + last;
}

__host__ __device__ inline int64_t run_cost(const Run& r) {
  return r.n > 0 ? cost_before(r, run_items(r)) : 0;
}

// The CTAs that work, and the shares [share_start(c), share_start(c + 1)).
__host__ __device__ inline int working_ctas(int64_t total, int grid) {
  const int64_t most = total / kMinShare;
  return most < 1 ? 1 : (most < grid ? static_cast<int>(most) : grid);
}
__host__ __device__ inline int64_t share_start(int64_t total, int ctas, int c) { return total * c / ctas; }
__host__ __device__ inline int share_owner(int64_t total, int ctas, int64_t pos) {
  return static_cast<int>(((pos + 1) * ctas - 1) / total);
}

// Key tiles [j0, j1) of an item at `start`, with w row tiles and n key tiles,
// that fall into the share [s0, s1).
__host__ __device__ inline void share_tiles(int64_t start, int w, int n, int64_t s0, int64_t s1, int* j0,
                                            int* j1) {
  const int64_t lo = s0 <= start ? 0 : (s0 - start + w - 1) / w;
  const int64_t hi = s1 <= start ? 0 : (s1 - start + w - 1) / w;
  *j0 = static_cast<int>(lo < n ? lo : n);
  *j1 = static_cast<int>(hi < n ? hi : n);
}

}  // namespace qspec
