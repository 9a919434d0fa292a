// How the attention of many tokens (prompt_attention.cuh) is shared out.
//
// A tile is 128 query rows by 128 keys.  The rows of a tile belong to one KV
// head: row r holds query head g * group + r % group of token r / group, so
// grouped heads fill the tile and share its keys.  An item is the work of one
// KV head on a run of at most 2 * tpt tokens (tpt = 128 / group, rounded
// down): two row tiles that share every key tile, or one when tpt tokens or
// fewer are left.  Items, in order:
//   a shared prefix taken once for all sequences: for g, for the runs of all packed tokens: its keys;
//   the sequences: for b, for g, for the runs of b's tokens: the keys that the run's last token sees
//   (behind those of the prefix where it is not taken for all together).
// An item costs (row tiles) x (key tiles) + kItemCost; the costs of all items
// laid end to end are cut into equal shares, one for each CTA, whatever the
// batch, the lengths and the heads.  A key tile belongs to the CTA in whose
// share its place on that line falls, so a long item is split over CTAs.
// Everything follows from the lengths in closed form (a sum of floors), so
// each CTA finds its share alone.
#pragma once

#include <cstdint>

namespace qspec {

constexpr int kItemCost = 2;       // an item's fixed cost (queries, output) in pairs of a row tile and a key tile
constexpr int kMinShare = 6;       // a CTA's smallest share: fewer CTAs work where there is less

// Unsigned division; 64 bits only where they are needed (a 64-bit division is a long software routine).
__host__ __device__ inline uint64_t div_u64(uint64_t a, uint64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// sum over i < n of floor((a i + b) / 128), for n, b < 2^31 and a <= 256: Euclid's steps on
// (a, 128).  After the first, which only shifts, every term but n is below 128.
__host__ __device__ inline int64_t floor_sum_128(int64_t n, int64_t a, int64_t b) {
  if (n <= 0) return 0;
  int64_t ans = (n - 1) * n / 2 * (a >> 7) + n * (b >> 7);
  a &= 127;
  uint64_t y = static_cast<uint64_t>(a) * n + (b & 127);
  if (y < 128) return ans;
  uint64_t m = a, k = y >> 7, c = y & 127, d = 128;     // sum over i < k of floor((d i + c) / m)
  for (;;) {
    const uint64_t qd = div_u64(d, m), qc = div_u64(c, m);
    ans += static_cast<int64_t>((k - 1) * k / 2 * qd + k * qc);
    d -= qd * m;
    c -= qc * m;
    y = d * k + c;
    if (y < m) return ans;
    k = div_u64(y, m);
    c = y - k * m;
    const uint64_t t = m;
    m = d;
    d = t;
  }
}

// The items of one KV head over a run of n tokens: all of them see the keys of
// `pre` key tiles first, then, where base >= 0, token t sees base + t + 1 keys of its own.
struct Run {
  int n;           // tokens
  int tpt;         // tokens of a row tile
  int base;        // own keys before the run's first token; < 0: no own keys
  int pre;         // key tiles that every token sees
};

__host__ __device__ inline int run_items(const Run& r) { return (r.n + 2 * r.tpt - 1) / (2 * r.tpt); }

__host__ __device__ inline int item_tokens(const Run& r, int i) {
  const int left = r.n - i * 2 * r.tpt;
  return left < 2 * r.tpt ? left : 2 * r.tpt;
}

// Key tiles that the first `tokens` tokens of item i see.
__host__ __device__ inline int item_tiles(const Run& r, int i, int tokens) {
  return r.pre + (r.base < 0 ? 0 : static_cast<int>((static_cast<uint32_t>(r.base) + i * 2 * r.tpt + tokens + 127u) >> 7));
}

__host__ __device__ inline int64_t cost_of(int row_tiles, int key_tiles) {
  return (row_tiles == 2 ? 2ll * key_tiles : key_tiles) + kItemCost;
}

// The cost of the items before item i (i <= run_items(r)).
__host__ __device__ inline int64_t cost_before(const Run& r, int i) {
  int64_t last = 0;
  if (i > 0) {
    const int tokens = item_tokens(r, i - 1);
    if (tokens < 2 * r.tpt) {                            // only a run's last item is not full
      --i;
      last = cost_of(tokens > r.tpt ? 2 : 1, item_tiles(r, i, tokens));
    }
  }
  const int64_t s = 2 * r.tpt;
  const int64_t own = r.base < 0 ? 0 : floor_sum_128(i, s, r.base + s + 127);
  return 2 * (own + static_cast<int64_t>(i) * r.pre) + static_cast<int64_t>(i) * kItemCost + last;
}

__host__ __device__ inline int64_t run_cost(const Run& r) {
  return r.n > 0 ? cost_before(r, run_items(r)) : 0;
}

// The CTAs that work, and the shares [share_start(c), share_start(c + 1)).
__host__ __device__ inline int working_ctas(int64_t total, int grid) {
  if (total >= static_cast<int64_t>(grid) * kMinShare) return grid;
  const int most = static_cast<int>(total) / kMinShare;
  return most < 1 ? 1 : most;
}
__host__ __device__ inline int64_t share_start(int64_t total, int ctas, int c) {
  return static_cast<int64_t>(div_u64(static_cast<uint64_t>(total) * c, ctas));
}
__host__ __device__ inline int share_owner(int64_t total, int ctas, int64_t pos) {
  return static_cast<int>(div_u64(static_cast<uint64_t>(pos + 1) * ctas - 1, total));
}

// Key tiles [j0, j1) of an item at `start`, with w row tiles and n key tiles,
// that fall into the share [s0, s1).
__host__ __device__ inline void share_tiles(int64_t start, int w, int n, int64_t s0, int64_t s1, int* j0,
                                            int* j1) {
  const int up = w - 1;                                  // w is 1 or 2: a shift divides
  const int64_t lo = s0 <= start ? 0 : (s0 - start + up) >> up;
  const int64_t hi = s1 <= start ? 0 : (s1 - start + up) >> up;
  *j0 = static_cast<int>(lo < n ? lo : n);
  *j1 = static_cast<int>(hi < n ? hi : n);
}

}  // namespace qspec
