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
// The costs of all items (below) laid end to end are cut into equal shares, one for each CTA, whatever the
// batch, the lengths and the heads.  A key tile belongs to the CTA in whose
// share its place on that line falls, so a long item is split over CTAs.
// Everything follows from the lengths in closed form (a sum of floors), so
// each CTA finds its share alone.
#pragma once

#include <cstdint>

namespace qspec {

// Costs, in units of about 850 cycles: a key tile for two row tiles or one, and what an item of either kind
// costs besides (queries, first scores, output).  Measured: 3450 and 2400 cycles for a tile, 7800 and 3900 for
// an item; other values, tried one by one, were no better.
constexpr int kTileCost2 = 4, kTileCost1 = 3, kItemCost2 = 8, kItemCost1 = 6;
constexpr int kMinShare = 12;      // a CTA's smallest share: fewer CTAs work where there is less

// Unsigned division; 64 bits only where they are needed (a 64-bit division is a long software routine).
__host__ __device__ inline uint64_t div_u64(uint64_t a, uint64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// sum over i < n of floor((s i + b) / 128), for n, b < 2^31 and 0 < s <= 256.
// Where s is a power of two (so are most groups of heads), shifts alone:
// below 128, floor((s i + b) / 128) = floor((i + floor(b / s)) / (128 / s)).
// Else Euclid's steps on (s, 128); after the first every term but n is below 128.
__host__ __device__ inline int64_t floor_sum_128(int64_t n, int s, int64_t b) {
  if (n <= 0) return 0;
  if ((s & (s - 1)) == 0) {
    if (s >= 128) return n * (b >> 7) + (s >> 7) * (n * (n - 1) / 2);
    int k = 0;                                           // 128 / s = 2^k
    while ((s << k) < 128) ++k;
    const int64_t e = b >> (7 - k), last = n + e;
    const int64_t q0 = e >> k, r0 = e - (q0 << k), q1 = last >> k, r1 = last - (q1 << k);
    return ((q1 * (q1 - 1) / 2) << k) + q1 * r1 - ((q0 * (q0 - 1) / 2) << k) - q0 * r0;
  }
  int64_t ans = (n - 1) * n / 2 * (s >> 7) + n * (b >> 7);
  const uint64_t a = s & 127;
  uint64_t y = a * n + (b & 127);
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

__host__ __device__ inline int run_items(const Run& r) {
  return r.n <= 2 * r.tpt ? (r.n > 0 ? 1 : 0) : (r.n + 2 * r.tpt - 1) / (2 * r.tpt);
}

__host__ __device__ inline int item_tokens(const Run& r, int i) {
  const int left = r.n - i * 2 * r.tpt;
  return left < 2 * r.tpt ? left : 2 * r.tpt;
}

// Key tiles that the first `tokens` tokens of item i see.
__host__ __device__ inline int item_tiles(const Run& r, int i, int tokens) {
  return r.pre + (r.base < 0 ? 0 : static_cast<int>((static_cast<uint32_t>(r.base) + i * 2 * r.tpt + tokens + 127u) >> 7));
}

__host__ __device__ inline int64_t cost_of(int row_tiles, int key_tiles) {
  return row_tiles == 2 ? static_cast<int64_t>(kTileCost2) * key_tiles + kItemCost2
                        : static_cast<int64_t>(kTileCost1) * key_tiles + kItemCost1;
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
  const int s = 2 * r.tpt;
  const int64_t own = r.base < 0 || i == 0 ? 0 : floor_sum_128(i, s, static_cast<int64_t>(r.base) + s + 127);
  return kTileCost2 * (own + static_cast<int64_t>(i) * r.pre) + static_cast<int64_t>(i) * kItemCost2 + last;
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
// (equal but for one unit, the larger ones first: one division for both ends)
__host__ __device__ inline void share_of(int64_t total, int ctas, int c, int64_t* s0, int64_t* s1) {
  const int64_t each = static_cast<int64_t>(div_u64(total, ctas));
  const int more = static_cast<int>(total - each * ctas);
  *s0 = each * c + (c < more ? c : more);
  *s1 = *s0 + each + (c < more ? 1 : 0);
}
__host__ __device__ inline int share_owner(int64_t total, int ctas, int64_t pos) {
  const int64_t each = static_cast<int64_t>(div_u64(total, ctas)), more = total - each * ctas;
  const int64_t large = more * (each + 1);
  return static_cast<int>(pos < large ? div_u64(pos, each + 1) : more + div_u64(pos - large, each));
}

// Key tiles [j0, j1) of an item at `start`, with n key tiles, that fall into the share [s0, s1).
__host__ __device__ inline void share_tiles(int64_t start, int row_tiles, int n, int64_t s0, int64_t s1, int* j0,
                                            int* j1) {
  const int64_t from = s0 <= start ? 0 : s0 - start, to = s1 <= start ? 0 : s1 - start;
  const int64_t all = static_cast<int64_t>(n) * (row_tiles == 2 ? kTileCost2 : kTileCost1);
  const uint64_t lo = from < all ? from : all, hi = to < all ? to : all;
  if (row_tiles == 2) {
    *j0 = static_cast<int>((lo + kTileCost2 - 1) / kTileCost2);
    *j1 = static_cast<int>((hi + kTileCost2 - 1) / kTileCost2);
  } else {
    *j0 = static_cast<int>((lo + kTileCost1 - 1) / kTileCost1);
    *j1 = static_cast<int>((hi + kTileCost1 - 1) / kTileCost1);
  }
}

}  // namespace qspec
