// Attention of many new tokens over the shared KV cache: packed causal
// prompts, and batches whose sequences share one prefix.
//
//   out_r = sum_j w_j v_j,  w = softmax_j(q_r . k_j / sqrt(128)) over the keys j that row r sees.
//
// One pass over the keys: for each tile of 128 keys S = Q K^T on the tensor
// cores, the running maximum m and sum l of the softmax in fp32 registers,
// P = exp(S - m) rounded to bf16 (its only rounding; the values are bf16, and
// both operands of the product have one type), O += P V in fp32 tensor
// memory, out = O / l (the running maximum and sum: Milakov and Gimelshein,
// 2018).  m is only raised, and O scaled, when a tile exceeds it by more than
// 2^kRaise: until then P is at most 2^kRaise, with the same relative rounding.
//
// A CTA per SM works through its share of the items (prompt_schedule.cuh).
//   warp 10: finds the share's items and passes them on (ring of 4);
//   warp 8: TMA of queries (ring of two tiles) and of key and value tiles
//           (ring of 4 x 32 KB);
//   warp 9: tcgen05.mma: S of the next step before P V of the current one;
//   warps 0-3, 4-7: the softmax of slots 0 and 1, a thread for each row.  A slot
//           is a tile of S, and of O, in tensor memory; P takes S's place;
//   warps 12-15: the output of an item, while the softmax is at the next;
//   warp 11: clears the rows of sequences that are refused.
// With two row tiles, each has a slot, and both use every key tile.  With one,
// the slots take alternate key tiles and are joined at the end of the item.
// A piece of a split item is left in the workspace as (m, l, O); a second
// kernel joins the pieces in order.
//
// What bounds it.  Long prompts (8192 tokens, 32 heads over 8: 506 us, 1.09 PFLOP/s in a burst; 571 us, 0.96
// in runs of a second, the power limit holding the clock at 1.7 GHz): a slot's chain of S (515 cycles),
// softmax (1600), P V (515) and their hand-overs, about 3300 cycles for a key tile of which the tensor cores
// work 2060 for both slots.  Single tokens: HBM, and the same chain.  Short prompts: the way to the first item
// (about 5 us) and HBM's answer to all CTAs' first loads.  Measured and not kept, being slower or no faster: two
// threads for each row, one pass over S with the maximum kept as a whole number, a third query tile, a fifth
// key tile, joining in this kernel.
#pragma once

#include <cuda_bf16.h>
#include <cstddef>
#include <cstdint>

#include "attention.cuh"
#include "device_common.cuh"
#include "prompt_rope.cuh"
#include "prompt_schedule.cuh"

namespace qspec {

constexpr int kPaStages = 4;
constexpr int kPaItems = 4;                                  // items passed on ahead
constexpr int kPaThreads = 512;
constexpr int kPaTileBytes = 128 * kHeadDim * 2;             // 32 KB: a tile of Q, K or V
constexpr float kScoreLog2 = kInvSqrtHeadDim * 1.4426950408889634f;   // scores in powers of two
constexpr float kRaise = 8.f;

// How a shared prefix is taken: once for the rows of all sequences together, or ahead of the own keys of each.
enum : int { kPaNoPrefix = 0, kPaPrefixOnce = 1, kPaPrefixAhead = 2 };
// With so many rows of a KV head in a sequence, on average, the prefix goes ahead of its own keys: 24
// sequences of 96 rows behind 3000 positions, 64 query heads over 8, 61 us (once for all: 64), of 256 rows 94
// (139); of 64 rows 60 (52), of 32 rows 57 (41).
constexpr int kPaAheadRows = 96;

struct PromptArgs {
  const int32_t* cu;           // null: t_new tokens for every sequence
  const int32_t* lens;
  const int32_t* prefix_len;   // null: no prefix
  uint16_t* out;
  uint8_t* work;
  int64_t ld_out;
  int64_t off_owners, off_desc, off_ml, off_o, off_row_ml, off_row_o;
  int n_tok, batch, t_new, offset, h_q, h_kv, group, tpt, l_max, prefix_max, mode;
  int ctas;                    // of the attention's grid
  int parts;                   // > 0: few items (and batch <= 32), each can have so many CTAs of its own
  uint32_t test_stall;         // test hook (0 = off), 1: the first key tile is never known to have landed
};

// A split item that ends in a CTA's share: its pieces are those of CTAs first .. this one.
struct PaJoin {
  int32_t valid, first, tok, tokens, g;
  int32_t refused;             // (CTA 0's) the starts are out of order: every row is zero already
  int32_t pad[2];
};

// Workspace: status word, what the GEMMs keep there, then per CTA two pieces of two row tiles
// (O in blocks of 4 columns: [32][128 rows][4]); with a prefix taken once, for the prefix and for own
// keys, by an item's first token and KV head, the CTAs that have its pieces (first, last), and for each
// (token, head) a whole row.
constexpr int64_t kPaOffDesc = 8192;
struct PaLayout {
  int64_t off_owners, off_desc, off_ml, off_o, off_row_ml, off_row_o, total;
};
__host__ __device__ inline PaLayout pa_layout(int64_t grid, int64_t kv_rows, int64_t rows, bool prefix) {
  PaLayout l;
  auto up = [](int64_t v) { return (v + 255) / 256 * 256; };
  l.off_desc = kPaOffDesc;
  l.off_ml = up(l.off_desc + grid * static_cast<int64_t>(sizeof(PaJoin)));
  l.off_o = up(l.off_ml + grid * 4 * 128 * 8);
  l.off_owners = up(l.off_o + grid * 4 * 128 * kHeadDim * 4);
  l.off_row_ml = up(l.off_owners + (prefix ? 2 * kv_rows * 8 : 0));
  l.off_row_o = up(l.off_row_ml + (prefix ? 2 * rows * 8 : 0));
  l.total = l.off_row_o + (prefix ? 2 * rows * kHeadDim * 4 : 0);
  return l;
}

// ---------------------------------------------------------------- instructions
// 32 lanes x 32 consecutive 32-bit columns (the counterpart of tmem_ld16).
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31"
      "}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
        "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
        "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t c0,
                                            int32_t c1, int32_t c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t c0,
                                            int32_t c1, int32_t c2, int32_t c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// D (tensor memory) (+)= A x B, both in shared memory.
__device__ __forceinline__ void mma_ss_bf16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Descriptor of a [K][N] operand whose rows run along N (values: keys x head
// columns) in 128-byte swizzled blocks of 64 columns: the blocks are 16 KB
// apart, groups of 8 keys 1024 bytes.
__device__ __forceinline__ uint64_t smem_desc_rows_n(uint32_t addr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((addr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(16384u >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}
constexpr uint32_t kIdescScores = idesc_bf16(128);
constexpr uint32_t kIdescValues = idesc_bf16(128) | (1u << 16);   // B's rows run along N

// A warp's bounded wait without a call: around a call the 128 scores of a row, or the tensor core
// warp's uniform registers, would have to be saved.
__device__ __forceinline__ bool pa_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, uint32_t* status) {
  uint64_t start = 0;
  bool ok = mbar_try_wait(bar, parity);
  while (!ok) {
    ok = mbar_try_wait_sleep(bar, parity, 20000u);
    if (ok) break;
    const uint64_t now = global_timer_ns();
    if (start == 0) start = now;
    if (*abort_flag || now - start > kWaitLimitNs) {
      if (!*abort_flag) atomicOr(status, kDevStopped);
      *abort_flag = 1;
      break;
    }
  }
  return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y), "f"(z.x), "f"(z.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
  return d;
}

// (subnormal terms and sums count as 0)
__device__ __forceinline__ float2 add2_ftz(float2 x, float2 y) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.ftz.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
  return d;
}

__device__ __forceinline__ float max3(float x, float y, float z) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(x), "f"(y), "f"(z));
  return d;
}
// The largest, or NaN where one of them is NaN.
__device__ __forceinline__ float max3_nan(float x, float y, float z) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(x), "f"(y), "f"(z));
  return d;
}
// One of so many pairs of weights comes from exp2_poly: the special function unit, at 4 a cycle for
// each quarter of an SM, takes 1024 cycles for a warp's tile alone.  Cycles for the weights of a tile,
// by the share of pairs: none 1400, an eighth 1200, a quarter 1060, three eighths 1190, half 1550.
constexpr int kPolyEach = 4;

// 2^x for x <= 2^7 without the special function unit (the reduction of Cody and
// Waite, 1980): x = k + r with k the nearest integer (by adding 1.5 x 2^23, whose
// last bits then hold k), 2^r by a polynomial, k added to its exponent.  The polynomial is the one of degree 3
// with the least relative error on |r| <= 1/2 (7.5e-5, from a weighted
// least-squares fit): 1/26 of half a step of the bf16 that its result becomes.
// x <= -126 (a key that is not seen has -inf) is taken as -126, whose power by the cubic, 0.99996 2^-126, is
// subnormal: the addition at the end makes it 0, as ex2 has it.  (Kept, such a weight brings 1.2 into the
// output for a value of 10^38 that the row does not see.)
__device__ __forceinline__ float2 exp2_poly(float2 x) {
  x.x = fmaxf(x.x, -126.f);
  x.y = fmaxf(x.y, -126.f);
  const float2 big = make_float2(12582912.f, 12582912.f), neg = make_float2(-12582912.f, -12582912.f);
  const float2 t = add2(x, big);
  const float2 k = add2(t, neg);
  const float2 r = fma2(k, make_float2(-1.f, -1.f), x);
  float2 y = fma2(r, make_float2(0x1.c3f760p-5f, 0x1.c3f760p-5f), make_float2(0x1.f0de1ap-3f, 0x1.f0de1ap-3f));
  y = fma2(y, r, make_float2(0x1.62f31ap-1f, 0x1.62f31ap-1f));
  y = fma2(y, r, make_float2(0x1.fff692p-1f, 0x1.fff692p-1f));
  y.x = __int_as_float((__float_as_int(t.x) << 23) + __float_as_int(y.x));
  y.y = __int_as_float((__float_as_int(t.y) << 23) + __float_as_int(y.y));
  return add2_ftz(y, make_float2(0.f, 0.f));
}

// ---------------------------------------------------------------- finding the items
// Sequence b's packed tokens and the keys before them; n = 0 where its
// offsets or its length are not those of the cache.  Where starts fall, a row could belong to two
// sequences (and be written by both): then the whole call is refused.
struct PaSequence {
  int tok0, n, base;
  bool bad, falls;             // falls: it ends before it starts
};
__device__ __forceinline__ PaSequence pa_sequence(const PromptArgs& a, int b) {
  PaSequence s;
  int n;
  s.bad = s.falls = false;
  const int64_t len = a.lens[b];
  if (a.cu) {
    s.tok0 = a.cu[b];
    const int end = a.cu[b + 1];
    s.falls = end < s.tok0;
    s.bad = s.tok0 < 0 || s.falls || end > a.n_tok;
    n = s.bad ? 0 : end - s.tok0;
  } else {
    s.tok0 = b * a.t_new;
    n = a.t_new;
  }
  const int64_t base = len + a.offset;
  s.bad = s.bad || len < 0 || base + n > a.l_max;
  s.n = s.bad ? 0 : n;
  s.base = s.bad ? 0 : static_cast<int>(base);
  return s;
}

// The tokens that take part in the items of a prefix taken once.
__device__ __forceinline__ int pa_packed_tokens(const PromptArgs& a) {
  if (!a.cu) return a.n_tok;
  const int end = a.cu[a.batch];
  return end < 0 ? 0 : (end > a.n_tok ? a.n_tok : end);
}

// The prefix's length; -1 where it is refused.
__device__ __forceinline__ int pa_prefix(const PromptArgs& a) {
  if (!a.prefix_len) return 0;
  const int p = *a.prefix_len;
  return p < 0 || p > a.prefix_max ? -1 : p;
}

__device__ __forceinline__ Run pa_prefix_run(const PromptArgs& a, int prefix) {
  Run r;
  r.n = prefix > 0 && a.mode == kPaPrefixOnce ? pa_packed_tokens(a) : 0;
  r.tpt = a.tpt;
  r.base = -1;
  r.pre = (prefix + 127) >> 7;
  return r;
}
__device__ __forceinline__ Run pa_own_run(const PromptArgs& a, const PaSequence& s, int prefix) {
  Run r;
  r.n = prefix < 0 ? 0 : s.n;
  r.tpt = a.tpt;
  r.base = s.base;
  r.pre = a.mode == kPaPrefixAhead ? (prefix + 127) >> 7 : 0;
  return r;
}

// An item, or what of it lies in this CTA's share, as the warps get it.
struct PaItem {
  int32_t tok, tokens;         // packed tokens; tokens = 0: no more items
  int32_t g, head;             // KV head; its place among the caches' heads
  int32_t j0, j1, end0;        // key tiles of the share; those that the first of two row tiles sees end at end0
  int32_t pre_tiles, pre;      // the first key tiles are the prefix's, with so many keys
  int32_t sees;                // own keys that the first token sees (each later one sees one more)
  int32_t flags, first_cta;
};
enum : int { kPaTwo = 1, kPaWhole = 2, kPaCarried = 4, kPaEnds = 8, kPaOnce = 16 };

struct PaShare {
  int64_t s0, s1, total;
  int64_t start;               // of the sequence in which the share begins
  int b, ctas;                 // b < 0: the prefix
  bool refused;
};

// Barriers and small exchanges in shared memory.
constexpr int kPaBarriers = 2 * kPaStages + 17 + 2 * kPaItems;
struct PaShared {
  uint64_t kv_full[kPaStages], kv_empty[kPaStages], q_full[2], q_empty[2];      // (initialised in this order)
  uint64_t s_ready[2], p_ready[2], pv_done[2], o_free[2], ml_full[2], ml_free[2], drained;
  uint64_t item_full[kPaItems], item_empty[kPaItems];
  PaItem items[kPaItems];
  PaShare share;
  int64_t warp_sums[kPaThreads / 32];
  int abort_flag;
  uint32_t tmem;
  float2 ml[2][128];
};
constexpr int kPaTilesBytes = (2 + kPaStages) * kPaTileBytes;          // Q, K and V tiles, then PaShared
constexpr int kPaSmemBytes = kPaTilesBytes + static_cast<int>(sizeof(PaShared));
static_assert(kPaSmemBytes <= 227 * 1024, "shared memory of a CTA");

// The last item of a run starting at `start` that starts at or before s0: [lo, lo + n) narrowed 32-fold
// by a warp; `at`: where it starts.
__device__ __noinline__ int64_t pa_cost_before(int n, int tpt, int base, int pre, int i) {
  Run r;
  r.n = n;
  r.tpt = tpt;
  r.base = base;
  r.pre = pre;
  return cost_before(r, i);
}
__device__ __forceinline__ int64_t pa_run_cost(const Run& r) {
  return r.n > 0 ? pa_cost_before(r.n, r.tpt, r.base, r.pre, run_items(r)) : 0;
}
__device__ __forceinline__ int pa_find_item(const Run& r, int64_t start, int64_t s0, int64_t* at) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = run_items(r);
  int64_t found = start;
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int64_t mine = start + (lane * step < n ? pa_cost_before(r.n, r.tpt, r.base, r.pre, lo + lane * step) : 0);
    const bool le = lane * step < n && (lane == 0 || mine <= s0);
    const int k = 31 - __clz(__ballot_sync(0xffffffffu, le));
    found = __shfl_sync(0xffffffffu, mine, k);
    lo += k * step;
    n = min(step, n - k * step);
  }
  *at = found;
  return lo;
}

constexpr int kPaWarpBatch = 64;     // up to so many sequences one warp finds the shares alone

// More sequences than that: the whole CTA sums their costs, and finds the one in which its share begins.
__device__ __forceinline__ void pa_find_share(const PromptArgs& a, PaShared& sm) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int prefix = pa_prefix(a);
  const int64_t prefix_all = pa_run_cost(pa_prefix_run(a, prefix)) * a.h_kv;
  int64_t before = prefix_all;         // the cost before the chunk of sequences at hand
  int64_t cost = 0, at = 0;            // of one KV head of this thread's sequence; before the sequence
  bool falls = false;
  auto scan = [&](int b) {
    cost = 0;
    if (b < a.batch) {
      const PaSequence s = pa_sequence(a, b);
      falls = falls || s.falls;
      cost = pa_run_cost(pa_own_run(a, s, prefix));
    }
    const int64_t mine = cost * a.h_kv;
    int64_t incl = mine;
#pragma unroll 1
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t o = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += o;
    }
    if (lane == 31) sm.warp_sums[warp] = incl;
    __syncthreads();
    int64_t all = 0;
    at = before + incl - mine;
#pragma unroll 1
    for (int k = 0; k < kPaThreads / 32; ++k) {
      const int64_t s = sm.warp_sums[k];
      if (k < warp) at += s;
      all += s;
    }
    before += all;
    __syncthreads();                   // the sums are written again
  };
#pragma unroll 1
  for (int b0 = 0; b0 < a.batch; b0 += kPaThreads) scan(b0 + tid);
  const bool refused = __syncthreads_or(falls);
  const int64_t total = refused ? 0 : before;
  const int ctas = working_ctas(total, gridDim.x), c = blockIdx.x;
  int64_t s0 = total, s1 = total;
  if (c < ctas && total > 0) share_of(total, ctas, c, &s0, &s1);
  if (tid == 0) {
    sm.share.s0 = s0;
    sm.share.s1 = s1;
    sm.share.total = total;
    sm.share.ctas = ctas;
    sm.share.b = -1;
    sm.share.start = 0;
    sm.share.refused = refused;
  }
  __syncthreads();
  before = prefix_all;
#pragma unroll 1
  for (int b0 = 0; b0 < a.batch; b0 += kPaThreads) {
    const int b = b0 + tid;
    if (a.batch > kPaThreads) scan(b);           // else this thread's values still stand
    if (b < a.batch) {
      if (cost > 0 && at <= s0 && s0 < at + cost * a.h_kv) {
        sm.share.b = b;
        sm.share.start = at;
      }
    }
  }
  __syncthreads();
}

// ---------------------------------------------------------------- the roles of the warps
// Few and short items (at most 32 sequences): each has a.parts CTAs of its own, and this one's item, or part
// of one (kPaMinPart key tiles at least), is found without the shares.  0: there is none for this CTA; -1: the
// longest item would keep its CTAs for more than kPaPartTiles tiles, so that the shares are better.
// us with 4, 6, 8, 12, 16 tiles at most (16 x 1 token behind 1000, 32 heads over 8): 26 26 21 21 21;
// 3 x 20 behind 4000, 64 over 8: 31 31 31 37 37.  With parts of 4, 3, 2 tiles at least: 64 tokens behind
// 1000 20.0 20.1 18.9, 4 x 1 behind a prefix of 500 15.7 13.9 13.9.
constexpr int kPaPartTiles = 8;
constexpr int kPaMinPart = 2;
__device__ __forceinline__ int pa_find_one(const PromptArgs& a, PaShared& sm, PaItem* it) {
  const int lane = threadIdx.x & 31;
  const int prefix = pa_prefix(a);
  PaSequence mine;
  mine.n = 0;
  mine.base = 0;
  mine.falls = false;
  if (lane < a.batch) mine = pa_sequence(a, lane);
  const bool refused = __any_sync(0xffffffffu, mine.falls);
  if (lane == 0) sm.share.refused = refused;
  if (refused) return 0;
  Run run = pa_prefix_run(a, prefix);
  const Run own = pa_own_run(a, mine, prefix);
  const int longest = max(run.n > 0 ? run.pre : 0,
                          __reduce_max_sync(0xffffffffu, own.n > 0 ? item_tiles(own, 0, own.n) : 0));
  if (longest > kPaPartTiles * a.parts) return -1;
  int k = blockIdx.x / a.parts, b = -1, tok0 = 0, items = run_items(run);
  const int part = blockIdx.x - k * a.parts;
  if (k >= items * a.h_kv) {
    k -= items * a.h_kv;
    const int each = run_items(own), all = each * a.h_kv;
    int incl = all;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += o;
    }
    const uint32_t after = __ballot_sync(0xffffffffu, k < incl);
    if (after == 0) return 0;
    b = __ffs(after) - 1;
    k -= __shfl_sync(0xffffffffu, incl - all, b);
    items = __shfl_sync(0xffffffffu, each, b);
    run.n = __shfl_sync(0xffffffffu, own.n, b);
    run.base = __shfl_sync(0xffffffffu, own.base, b);
    run.pre = own.pre;
    tok0 = __shfl_sync(0xffffffffu, mine.tok0, b);
  }
  const int g = items == 1 ? k : k / items, i = items == 1 ? 0 : k - g * items;
  const int tokens = item_tokens(run, i), n = item_tiles(run, i, tokens), w = tokens > run.tpt ? 2 : 1;
  const int parts = min(a.parts, (n + kPaMinPart - 1) / kPaMinPart);
  if (part >= parts) return 0;
  const int first = i * 2 * run.tpt;
  it->tok = tok0 + first;
  it->tokens = tokens;
  it->g = g;
  it->head = b < 0 ? g : b * a.h_kv + g;
  it->j0 = parts == 1 ? 0 : static_cast<int>(static_cast<int64_t>(n) * part / parts);
  it->j1 = parts == 1 ? n : static_cast<int>(static_cast<int64_t>(n) * (part + 1) / parts);
  it->end0 = w == 1 ? it->j1 : min(it->j1, max(it->j0, item_tiles(run, i, run.tpt)));
  it->pre_tiles = run.pre;
  it->pre = prefix;
  it->sees = run.base + first + 1;
  it->flags = (w == 2 ? kPaTwo : 0) | (parts == 1 ? kPaWhole : 0) | (part > 0 ? kPaCarried : 0) |
              (part == parts - 1 ? kPaEnds : 0) | (b < 0 ? kPaOnce : 0);
  it->first_cta = static_cast<int>(blockIdx.x) - part;
  if (a.mode == kPaPrefixOnce && part == 0 && lane == 0) {
    const int64_t at = (b < 0 ? 0 : static_cast<int64_t>(a.n_tok) * a.h_kv) + static_cast<int64_t>(it->tok) * a.h_kv + g;
    reinterpret_cast<int2*>(a.work + a.off_owners)[at] = make_int2(it->first_cta, it->first_cta + parts - 1);
  }
  return 1;
}

// Passes an item on (its number `count` in the CTA).
__device__ __forceinline__ bool pa_pass(PaShared& sm, const PaItem& it, uint32_t count, uint32_t* status) {
  const uint32_t slot = count % kPaItems;
  if (!pa_wait(smem_u32(&sm.item_empty[slot]), ((count / kPaItems) & 1) ^ 1, &sm.abort_flag, status)) return false;
  if ((threadIdx.x & 31) == 0) {
    sm.items[slot] = it;
    mbar_arrive(smem_u32(&sm.item_full[slot]));
  }
  __syncwarp();
  return true;
}

// Warp 10: the share's items in order, into the ring.
__device__ __forceinline__ void pa_find_items(const PromptArgs& a, PaShared& sm) {
  const int lane = threadIdx.x & 31;
  uint32_t* const status = reinterpret_cast<uint32_t*>(a.work);
  if (a.parts > 0) {
    PaItem one;
    const int there = pa_find_one(a, sm, &one);
    if (there >= 0) {
      __syncthreads();           // the barriers are there (the other warps have waited for this one)
      if (there) pa_pass(sm, one, 0, status);
      one.tokens = 0;
      pa_pass(sm, one, there, status);
      return;
    }
  }
  const int prefix = pa_prefix(a);
  const Run prefix_run = pa_prefix_run(a, prefix);
  const int64_t prefix_head = pa_run_cost(prefix_run);
  PaSequence mine;               // of sequence block * 32 + lane
  int b = -1, block = -1;
  int64_t total, s0, s1, start = 0, head_cost = prefix_head;
  int ctas;
  bool falls = false;
  auto load = [&](int at) {
    if (at == block) return;
    block = at;
    mine.n = 0;
    mine.falls = false;
    if (block * 32 + lane < a.batch) mine = pa_sequence(a, block * 32 + lane);
  };
  auto own_run = [&](int of) -> Run {
    PaSequence s;
    s.n = __shfl_sync(0xffffffffu, mine.n, of & 31);
    s.base = __shfl_sync(0xffffffffu, mine.base, of & 31);
    return pa_own_run(a, s, prefix);
  };
  if (a.batch <= kPaWarpBatch) {
    // every lane: the cost of a sequence, or of two; then which of them the share begins in
    int64_t cost[2] = {0, 0}, at[2] = {0, 0};
    total = prefix_head * a.h_kv;
#pragma unroll 1
    for (int half = 1; half >= 0; --half) {       // the first 32 last: they stay in `mine`
      if (half * 32 >= a.batch) continue;
      load(half);
      falls = falls || mine.falls;
      const int64_t one = pa_run_cost(pa_own_run(a, mine, prefix));
      int64_t incl = one * a.h_kv;
#pragma unroll 1
      for (int off = 1; off < 32; off <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += o;
      }
      if (half == 0) {
        cost[0] = one;
        at[0] = prefix_head * a.h_kv + incl - one * a.h_kv;
        const int64_t sum = __shfl_sync(0xffffffffu, incl, 31);
        at[1] += prefix_head * a.h_kv + sum;
        total += sum;
      } else {
        cost[1] = one;
        at[1] = incl - one * a.h_kv;
        total += __shfl_sync(0xffffffffu, incl, 31);
      }
    }
    falls = __any_sync(0xffffffffu, falls);
    if (lane == 0) sm.share.refused = falls;
    if (falls) total = 0;
    ctas = working_ctas(total, gridDim.x);
    s0 = s1 = total;
    if (blockIdx.x < ctas && total > 0) share_of(total, ctas, blockIdx.x, &s0, &s1);
    const uint32_t in0 = __ballot_sync(0xffffffffu, cost[0] > 0 && at[0] <= s0 && s0 < at[0] + cost[0] * a.h_kv);
    const uint32_t in1 = __ballot_sync(0xffffffffu, cost[1] > 0 && at[1] <= s0 && s0 < at[1] + cost[1] * a.h_kv);
    if (in0 | in1) {
      const int of = __ffs(in0 ? in0 : in1) - 1;
      b = of + (in0 ? 0 : 32);
      start = __shfl_sync(0xffffffffu, in0 ? at[0] : at[1], of);
      head_cost = __shfl_sync(0xffffffffu, in0 ? cost[0] : cost[1], of);
    }
  } else {
    total = sm.share.total;
    ctas = sm.share.ctas;
    s0 = sm.share.s0;
    s1 = sm.share.s1;
    b = sm.share.b;
    start = sm.share.start;
    if (b >= 0) {
      load(b >> 5);
      head_cost = pa_run_cost(own_run(b));
    }
  }
  PaItem it;
  Run run = prefix_run;
  int tok0 = 0, i = 0, g = 0;
  if (s0 < s1) {
    if (b >= 0) {
      load(b >> 5);
      run = own_run(b);
      tok0 = __shfl_sync(0xffffffffu, mine.tok0, b & 31);
    }
    if (s0 > start) {
      if (s0 - start >= head_cost) {
        g = static_cast<int>(div_u64(s0 - start, head_cost));
        start += g * head_cost;
      }
      i = pa_find_item(run, start, s0, &start);
    }
  }
  if (a.batch <= kPaWarpBatch) __syncthreads();   // the barriers are there (the other warps have waited for this one)
  uint32_t count = 0;
  if (s0 < s1) {
    int items = run_items(run);
#pragma unroll 1
    while (start < s1) {
      const int tokens = item_tokens(run, i);
      const int w = tokens > run.tpt ? 2 : 1;
      const int n = item_tiles(run, i, tokens);
      share_tiles(start, w, n, s0, s1, &it.j0, &it.j1);
      if (it.j0 < it.j1) {
        const int first = i * 2 * run.tpt;
        it.tok = tok0 + first;
        it.tokens = tokens;
        it.g = g;
        it.head = b < 0 ? g : b * a.h_kv + g;
        it.end0 = w == 1 ? it.j1 : min(it.j1, max(it.j0, item_tiles(run, i, run.tpt)));
        it.pre_tiles = run.pre;
        it.pre = prefix;
        it.sees = run.base + first + 1;
        const bool whole = it.j0 == 0 && it.j1 == n;
        it.flags = (w == 2 ? kPaTwo : 0) | (whole ? kPaWhole : 0) | (start < s0 ? kPaCarried : 0) |
                   (it.j1 == n ? kPaEnds : 0) | (b < 0 ? kPaOnce : 0);
        it.first_cta = start < s0 ? share_owner(total, ctas, start) : blockIdx.x;
        if (a.mode == kPaPrefixOnce && it.j0 == 0) {
          const int64_t end = start + static_cast<int64_t>(w == 2 ? kTileCost2 : kTileCost1) * (n - 1);
          const int last = whole ? blockIdx.x : share_owner(total, ctas, end);
          const int64_t at = (b < 0 ? 0 : static_cast<int64_t>(a.n_tok) * a.h_kv) + static_cast<int64_t>(it.tok) * a.h_kv + g;
          if (lane == 0) reinterpret_cast<int2*>(a.work + a.off_owners)[at] = make_int2(blockIdx.x, last);
        }
        if (!pa_pass(sm, it, count++, status)) return;
      }
      start += cost_of(w, n);
      if (++i >= items) {
        i = 0;
        if (++g >= a.h_kv) {
          g = 0;
          do {
            if (++b >= a.batch) break;
            load(b >> 5);
            run = own_run(b);
          } while (run.n == 0);
          if (b >= a.batch) break;
          tok0 = __shfl_sync(0xffffffffu, mine.tok0, b & 31);
          items = run_items(run);
        }
      }
    }
  }
  it.tokens = 0;
  pa_pass(sm, it, count, status);
}

// Waits for item `count` of the ring; its readers say when they have it.
__device__ __forceinline__ bool pa_item_wait(PaShared& sm, uint32_t count, uint32_t* status) {
  return pa_wait(smem_u32(&sm.item_full[count % kPaItems]), (count / kPaItems) & 1, &sm.abort_flag, status);
}

// Warp 8: loads.
__device__ __forceinline__ void pa_load(const PromptArgs& a, PaShared& sm, uint32_t q_s, uint32_t kv_s,
                                        const CUtensorMap* tm_q, const CUtensorMap* tm_k, const CUtensorMap* tm_v,
                                        const CUtensorMap* tm_pk, const CUtensorMap* tm_pv) {
  uint32_t* const status = reinterpret_cast<uint32_t*>(a.work);
  volatile int* const abort_flag = &sm.abort_flag;
  const uint32_t leader = elect_one_lane();
  uint32_t ring = 0, qn = 0;
  bool ok = true;
  for (uint32_t count = 0;; ++count) {
    ok = pa_item_wait(sm, count, status);
    if (!ok) break;
    const PaItem it = sm.items[count % kPaItems];
    __syncwarp();
    if (leader) mbar_arrive(smem_u32(&sm.item_empty[count % kPaItems]));
    if (it.tokens == 0) break;
    const bool two = it.flags & kPaTwo;
    // (a first row tile that sees none of the share's keys is left out)
    for (int x = two && it.end0 == it.j0 ? 1 : 0; x < (two ? 2 : 1) && ok; ++x) {
      const uint32_t slot = qn & 1;
      ok = pa_wait(smem_u32(&sm.q_empty[slot]), ((qn >> 1) & 1) ^ 1, abort_flag, status);
      if (!ok) break;
      if (leader) {
        const uint32_t bar = smem_u32(&sm.q_full[slot]);
        const uint32_t dst = q_s + slot * kPaTileBytes;
        mbar_arrive_expect_tx(bar, static_cast<uint32_t>(a.tpt * a.group) * kHeadDim * 2);
        tma_load_3d(dst, tm_q, bar, 0, it.g * a.group, it.tok + x * a.tpt);
        tma_load_3d(dst + kPaTileBytes / 2, tm_q, bar, 64, it.g * a.group, it.tok + x * a.tpt);
      }
      ++qn;
    }
    for (int j = it.j0; j < it.j1 && ok; ++j) {
      const bool pre = j < it.pre_tiles;
      const int row = (pre ? j : j - it.pre_tiles) * 128;
      const int head = pre ? it.g : it.head;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const uint32_t st = ring % kPaStages;
        ok = ok && pa_wait(smem_u32(&sm.kv_empty[st]), ((ring / kPaStages) & 1) ^ 1, abort_flag, status);
        if (!ok) break;
        if (leader) {
          const uint32_t bar = smem_u32(&sm.kv_full[st]);
          mbar_arrive_expect_tx(bar, kPaTileBytes);
          tma_load_4d(kv_s + st * kPaTileBytes, kv ? (pre ? tm_pv : tm_v) : (pre ? tm_pk : tm_k), bar, 0, row, 0, head);
        }
        ++ring;
      }
    }
    if (!ok) break;
  }
  if (!ok) {
    // given up: let the copies in flight land before shared memory goes
    for (uint32_t r = ring > kPaStages ? ring - kPaStages : 0; r < ring; ++r)
      mbar_wait_drain(smem_u32(&sm.kv_full[r % kPaStages]), (r / kPaStages) & 1);
    for (uint32_t r = qn > 2 ? qn - 2 : 0; r < qn; ++r)
      mbar_wait_drain(smem_u32(&sm.q_full[r & 1]), (r >> 1) & 1);
  }
}

// Warp 9: tensor cores.  A step is one key tile in one slot: S, and when the softmax has made P of it,
// P V.  While a slot's softmax runs, the other slot's products do: S of the next step is issued before
// P V of the current one where its keys are there.  The queue of the tensor cores holds about two
// instructions, so what this warp does between them counts: a barrier that is complete costs 50 cycles
// to look at, a commit 60, a fence 65, against 1030 for the 16 products of a step.  Values that the
// instructions take are kept visibly the same for the whole warp (uniform registers), and P V is
// committed for the softmax at the end of the item alone: S of the same slot comes after it, and S's
// commit says that it is done.
// Each kind of product stands in the code once: the roles of the warps share the instruction caches, and
// what runs once an item is read from afar each time (with ten copies a short item took 12000 cycles).
__device__ __forceinline__ void pa_multiply(const PromptArgs& a, PaShared& sm, uint32_t tmem_v, uint32_t q_s, uint32_t kv_s) {
  const int lane = threadIdx.x & 31;
  uint32_t* const status = reinterpret_cast<uint32_t*>(a.work);
  volatile int* const abort_flag = &sm.abort_flag;
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_v, 0);
  bool ok = true, more = true, in_item = false;
  // the item at hand
  int j0 = 0, j1 = 0, end0 = 0, pre_tiles = 0, pre = 0, last_sees = 0;
  bool two = false, has0 = false;
  uint32_t count = 0;                        // items taken
  uint32_t qn = 0, singles = 0;              // query tiles, steps of items with one row tile
  // the ring place of the next S's keys (its values are in the next place), and the phase of its barrier
  uint32_t k_st = 0, k_ph = 0;
  auto forth = [](uint32_t& st, uint32_t& ph, uint32_t by) {
    st += by;
    if (st >= kPaStages) {
      st -= kPaStages;
      ph ^= 1;
    }
  };
  // the next S: its slot and queries, whether these and the keys are not known to have landed
  int j = 0;
  uint32_t slot = 0, q = 0;
  bool new_q = false, new_k = false;
  // P V to come of either slot: tail, ring place, phase, flags; which comes first
  constexpr uint32_t kStage = 256, kPhase = 2048, kFirst = 4096, kFree = 8192, kLast = 16384, kNew = 32768, kHave = 65536;
  uint32_t e0 = 0, e1 = 0, oldest = 0;
  uint32_t p_count = 0;                      // phases of p_ready: slot 0 in bit 0, slot 1 in bit 1
  uint32_t o_count0 = 0, o_count1 = 0;       // items with steps in the slots
  auto tail_of = [&](int t) -> int {         // keys seen of tile t and those after it
    return t < pre_tiles ? pre - t * 128 : last_sees - (t - pre_tiles) * 128;
  };
  const uint32_t kv_full = smem_u32(&sm.kv_full[0]), kv_empty = smem_u32(&sm.kv_empty[0]);
  while (ok) {
    if (!in_item && more) {
      const uint32_t bar = smem_u32(&sm.item_full[count % kPaItems]), ph = (count / kPaItems) & 1;
      bool got = __all_sync(0xffffffffu, mbar_test_wait(bar, ph));
      if (!got && !((e0 | e1) & kHave)) {
        ok = got = pa_wait(bar, ph, abort_flag, status);
        if (!ok) break;
      }
      if (got) {
        const int mine = lane < 12 ? reinterpret_cast<const int32_t*>(&sm.items[count % kPaItems])[lane] : 0;
        const int tokens = __shfl_sync(0xffffffffu, mine, 1);
        j0 = __shfl_sync(0xffffffffu, mine, 4);
        j1 = __shfl_sync(0xffffffffu, mine, 5);
        end0 = __shfl_sync(0xffffffffu, mine, 6);
        pre_tiles = __shfl_sync(0xffffffffu, mine, 7);
        pre = __shfl_sync(0xffffffffu, mine, 8);
        last_sees = __shfl_sync(0xffffffffu, mine, 9) + tokens - 1;
        two = __shfl_sync(0xffffffffu, mine, 10) & kPaTwo;
        if (elect_one_lane()) mbar_arrive(smem_u32(&sm.item_empty[count % kPaItems]));
        ++count;
        more = tokens != 0;
        in_item = more;
        has0 = two && end0 > j0;
        j = j0;
        slot = two ? (has0 ? 0 : 1) : singles & 1;
        q = qn;
        new_q = new_k = true;
      }
    }
    const uint32_t of_slot = slot ? e1 : e0, of_other = slot ? e0 : e1;
    if (in_item && !(of_slot & kHave)) {
      const uint32_t kb = kv_full + 8 * k_st;
      const uint32_t qb = smem_u32(&sm.q_full[q & 1]), qp = (q >> 1) & 1;
      bool ready = true;
      if (new_q | new_k) {
        ready = __all_sync(0xffffffffu, (!new_q || mbar_test_wait(qb, qp)) && (!new_k || mbar_test_wait(kb, k_ph)));
        if (!ready && !(of_other & kHave)) {
          ok = ready = pa_wait(qb, qp, abort_flag, status) && pa_wait(kb, k_ph, abort_flag, status);
          if (!ok) break;
        }
      }
      if (ready) {
        // the last step on this key tile, and on these queries
        const bool free_k = !two || slot == 1, free_q = j + 1 == (two && slot == 0 ? end0 : j1);
        const uint64_t q_desc = smem_desc_sw128(q_s + (q & 1) * kPaTileBytes);
        const uint64_t k_desc = smem_desc_sw128(kv_s + k_st * kPaTileBytes);
        if (elect_one_lane()) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint32_t off = ((k >> 2) * (kPaTileBytes / 2) + (k & 3) * 32) >> 4;
            mma_ss_bf16(tmem + slot * 128, q_desc + off, k_desc + off, kIdescScores, k > 0);
          }
          mma_commit(smem_u32(&sm.s_ready[slot]));
          if (free_k) mma_commit(kv_empty + 8 * k_st);
          if (free_q) mma_commit(smem_u32(&sm.q_empty[q & 1]));
        }
        __syncwarp();
        uint32_t v_st = k_st, v_ph = k_ph;
        forth(v_st, v_ph, 1);
        const uint32_t e = kHave | static_cast<uint32_t>(min(tail_of(j), 128)) | v_st * kStage | v_ph * kPhase |
                           (j == j0 || (!two && j == j0 + 1) ? kFirst : 0) | (free_k ? kFree : 0) |
                           ((two ? free_q : j + 2 >= j1) ? kLast : 0) | (new_k ? kNew : 0);
        if (!(of_other & kHave)) oldest = slot;
        if (slot) e1 = e; else e0 = e;
        // the next step
        new_k = free_k;
        new_q = two && j == j0 && slot == 0;
        if (two && slot == 0) {
          slot = 1;
          q = qn + 1;
        } else {
          forth(k_st, k_ph, 2);
          if (++j >= j1) {
            in_item = false;
            qn += has0 ? 2 : 1;
            if (!two) singles += j1 - j0;
          } else if (two) {
            slot = j < end0 ? 0 : 1;
            q = qn + (slot & (has0 ? 1 : 0));
          } else {
            slot ^= 1;
          }
        }
        continue;
      }
    }
    if (!((e0 | e1) & kHave)) {
      if (more) continue;
      break;
    }
    if (two && in_item && (e0 & e1 & kHave) && slot == 0 && oldest == 0 && !(e0 & (kFirst | kLast)) &&
        j + 1 < end0 && (j - 1 >= pre_tiles || j * 128 <= pre)) {
      // The middle of an item with two row tiles, all keys seen (neither is P V to come the last of an item):
      // nothing to decide but whether the keys are there.  P V of tile j - 1 and S of tile j, for slot 0,
      // then for slot 1.
      bool landed = true;
      // A barrier is looked at, and a fence made, while the last two products before are still queued.
      const uint32_t p0 = smem_u32(&sm.p_ready[0]), p1 = smem_u32(&sm.p_ready[1]);
      bool p_there = false;                    // P of the slot at hand is known (and fenced)
      uint32_t v_st = (e0 / kStage) & 7, v_ph = (e0 / kPhase) & 1;
      do {
        const uint32_t kb = kv_full + 8 * k_st;
        const uint64_t k_desc = smem_desc_sw128(kv_s + k_st * kPaTileBytes);
        const uint64_t v_desc = smem_desc_rows_n(kv_s + v_st * kPaTileBytes);
        if (!pa_wait(kv_full + 8 * v_st, v_ph, abort_flag, status)) { ok = false; break; }
#pragma unroll 1
        for (uint32_t x = 0; x < 2; ++x) {
          if (!p_there) {
            if (!pa_wait(x ? p1 : p0, (p_count >> x) & 1, abort_flag, status)) { ok = false; break; }
            tc_fence_after();
          }
          p_there = false;
          p_count ^= 1u << x;
          const uint64_t q_desc = smem_desc_sw128(q_s + ((qn + x) & 1) * kPaTileBytes);
          if (elect_one_lane()) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              mma_ts<false>(tmem + 256 + x * 128, tmem + x * 128 + k * 8, v_desc + k * (2048 >> 4), kIdescValues, 1);
            if (x) mma_commit(kv_empty + 8 * v_st);
          }
          __syncwarp();
          if (x == 0) {
            landed = __all_sync(0xffffffffu, mbar_test_wait(kb, k_ph));
            if (!landed) break;
          }
          if (elect_one_lane()) {
#pragma unroll
            for (int k = 0; k < 6; ++k) {
              const uint32_t off = ((k >> 2) * (kPaTileBytes / 2) + (k & 3) * 32) >> 4;
              mma_ss_bf16(tmem + x * 128, q_desc + off, k_desc + off, kIdescScores, k > 0);
            }
          }
          __syncwarp();
          p_there = __all_sync(0xffffffffu, mbar_test_wait(x ? p0 : p1, (p_count >> (x ^ 1)) & 1));
          if (p_there) tc_fence_after();
          if (elect_one_lane()) {
#pragma unroll
            for (int k = 6; k < 8; ++k) {
              const uint32_t off = ((k >> 2) * (kPaTileBytes / 2) + (k & 3) * 32) >> 4;
              mma_ss_bf16(tmem + x * 128, q_desc + off, k_desc + off, kIdescScores, 1);
            }
            mma_commit(smem_u32(&sm.s_ready[x]));
            if (x) mma_commit(kv_empty + 8 * k_st);
          }
          __syncwarp();
        }
        if (!ok || !landed) break;
        v_st = k_st;
        v_ph = k_ph;
        forth(v_st, v_ph, 1);
        forth(k_st, k_ph, 2);
        ++j;
      } while (j + 1 < end0 && (j - 1 >= pre_tiles || j * 128 <= pre));
      if (!ok) break;
      // tile j - 1 may be the prefix's last
      const uint32_t e = kHave | static_cast<uint32_t>(min(tail_of(j - 1), 128)) | v_st * kStage | v_ph * kPhase;
      e0 = e | kNew;
      e1 = e | kFree;
      if (!landed) {                           // P V of slot 0 is done, that of slot 1 is to come
        e0 = 0;
        oldest = 1;
        continue;
      }
    }
    // O (+)= P V of the oldest S
    const uint32_t ps = oldest, e = ps ? e1 : e0;
    if (ps) e1 = 0; else e0 = 0;
    oldest ^= 1;
    const int tail = e & 255;                  // the tile's first unseen key (128: none)
    const uint32_t v_st = (e / kStage) & 7;
    const uint32_t va = kv_s + v_st * kPaTileBytes;
    if ((e & kNew) && !pa_wait(kv_full + 8 * v_st, (e / kPhase) & 1, abort_flag, status)) { ok = false; break; }
    if (e & kFirst) {                          // the item before with steps in the slot has read its O
      const uint32_t before = ps ? o_count1++ : o_count0++;
      if (before > 0 && !pa_wait(smem_u32(&sm.o_free[ps]), (before - 1) & 1, abort_flag, status)) { ok = false; break; }
    }
    const int pv_steps = (tail + 15) >> 4;
    if (tail & 15) {
      // keys past the last one seen may hold anything: their weights are 0, their values are made 0
#pragma unroll 1
      for (int z = lane; z < (pv_steps * 16 - tail) * 16; z += 32) {
        const uint32_t at = va + ((z >> 3) & 1) * (kPaTileBytes / 2) + (tail + (z >> 4)) * 128 + (z & 7) * 16;
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0) : "memory");
      }
      fence_proxy_async_smem();
      __syncwarp();
    }
    if (!pa_wait(smem_u32(&sm.p_ready[ps]), (p_count >> ps) & 1, abort_flag, status)) { ok = false; break; }
    p_count ^= 1u << ps;
    tc_fence_after();
    const uint64_t v_desc = smem_desc_rows_n(va);
    if (elect_one_lane()) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < pv_steps)
          mma_ts<false>(tmem + 256 + ps * 128, tmem + ps * 128 + k * 8, v_desc + k * (2048 >> 4), kIdescValues,
                        k > 0 || !(e & kFirst));
      if (e & kFree) mma_commit(kv_empty + 8 * v_st);
      if (e & kLast) mma_commit(smem_u32(&sm.pv_done[ps]));
    }
    __syncwarp();
  }
  if (!ok) {
    // given up: the products in flight end before tensor memory goes
    if (elect_one_lane()) mma_commit(smem_u32(&sm.drained));
    __syncwarp();
    mbar_wait_drain(smem_u32(&sm.drained), 0);
  }
}

// Among the four lanes of a quad, unit j (16 bytes) of lane i goes to lane j's place i.
__device__ __forceinline__ void transpose_quad(uint32_t (&u)[16]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int bit = 2; bit >= 1; bit >>= 1) {
    const bool up = lane & bit;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k & bit) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t lo = u[k * 4 + e], hi = u[(k + bit) * 4 + e];
        const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? lo : hi, bit);
        if (up) u[k * 4 + e] = got; else u[(k + bit) * 4 + e] = got;
      }
    }
  }
}

// Warps 0-7: the softmax.
__device__ __forceinline__ void pa_softmax(const PromptArgs& a, PaShared& sm, uint32_t tmem) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t* const status = reinterpret_cast<uint32_t*>(a.work);
  volatile int* const abort_flag = &sm.abort_flag;
  const uint32_t slot = warp >> 2;
  const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;       // lane base of this warp, in bits 16..
  const int row = (warp & 3) * 32 + lane;
  const uint32_t s_t = tmem + slot * 128 + lanes, o_t = tmem + 256 + slot * 128 + lanes;
  const int row_tok = row / a.group;
  const uint32_t s_bar = smem_u32(&sm.s_ready[slot]), p_bar = smem_u32(&sm.p_ready[slot]);
  uint32_t own_steps = 0;                    // of this slot so far
  uint32_t own_items = 0;                    // items with steps in this slot
  uint32_t single_steps = 0;
  bool ok = true;
  for (uint32_t count = 0;; ++count) {
    if (!pa_item_wait(sm, count, status)) break;
    const PaItem& item = sm.items[count % kPaItems];
    const int tokens = item.tokens;
    if (tokens == 0) break;
    const bool two = item.flags & kPaTwo;
    const int j0 = item.j0, j1 = item.j1, end0 = item.end0, pre_tiles = item.pre_tiles;
    // this row: its token, and the keys that it sees
    const int x = two ? static_cast<int>(slot) : 0;                   // this thread's row tile
    const int tok_in_item = x * a.tpt + row_tok;
    const bool live = row_tok < a.tpt && tok_in_item < tokens;
    const int pre_sees = item.pre, own_sees = item.sees + tok_in_item;
    const int own_least = __shfl_sync(0xffffffffu, own_sees, 0);      // rows see more and more
    const bool warp_live = __any_sync(0xffffffffu, live);
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sm.item_empty[count % kPaItems]));
    const uint32_t turn = (slot ^ single_steps) & 1;                  // one row tile: which alternate key tiles
    int j = j0, step = 1, end = slot == 0 ? end0 : j1;
    if (!two) {
      j = j0 + turn;
      step = 2;
      end = j1;
      single_steps += j1 - j0;
    }
    if (j >= end) continue;                                           // no key tile for this slot
    float m = -INFINITY, l = 0.f;
    bool fresh = true;
    for (; j < end; j += step) {
      if (!pa_wait(s_bar, own_steps & 1, abort_flag, status)) { ok = false; break; }
      if (warp_live) {
        tc_fence_after();
        const bool in_pre = j < pre_tiles;
        const int at = (in_pre ? j : j - pre_tiles) * 128;
        const bool partly = at + 128 > (in_pre ? pre_sees : own_least);   // some key of the tile is not seen
        const int lim = (in_pre ? pre_sees : own_sees) - at;
        // Columns from `seen` on no row of the warp sees: neither read nor weighed, their P is 0.  Before
        // that, where some row does not see some column, -inf goes into S (a small loop for what is rare:
        // the warps of all roles share the instruction caches).
        int seen = 128;
        if (partly) {
          seen = __reduce_max_sync(0xffffffffu, max(min(lim, 128), 0));
#pragma unroll 1
          for (int c = max(0, __reduce_min_sync(0xffffffffu, lim)) & ~15; c < ((seen + 63) & ~63); c += 16) {
            uint32_t x[16];
            tmem_ld16(s_t + c, x);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = c + e < lim ? x[e] : 0xff800000u;
            tmem_st16(s_t + c, x);
          }
          tmem_st_wait();
        }
        // S is read twice, 32 columns at a time, in loops that stay small
        uint32_t u[2][32];
        float top = m;
        auto largest = [&](const uint32_t* x) {
          float t[2] = {top, -INFINITY};
#pragma unroll
          for (int e = 0; e < 32; e += 2) t[(e >> 1) & 1] = max3_nan(t[(e >> 1) & 1], __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
          top = max3_nan(t[0], t[1], t[1]);
        };
        tmem_ld32(s_t, u[0]);
#pragma unroll 1
        for (int c = 0; c < seen; c += 64) {
          tmem_ld_wait();
          tmem_ld32(s_t + c + 32, u[1]);
          largest(u[0]);
          tmem_ld_wait();
          if (c + 64 < seen) tmem_ld32(s_t + 64, u[0]);
          largest(u[1]);
        }
        tmem_ld_wait();
        tmem_ld32(s_t, u[0]);
        // (a score of NaN or +inf makes the row's maximum, and with it all of the row, NaN)
        const bool raise = live && top != -INFINITY && !((top - m) * kScoreLog2 <= kRaise);
        float f = 1.f;
        if (__any_sync(0xffffffffu, raise)) {
          if (top == INFINITY) top = NAN;
          f = raise ? ex2((m - top) * kScoreLog2) : 1.f;
          l *= f;
          if (raise) m = top;
        }
        const float mc = m == -INFINITY ? 0.f : -m * kScoreLog2;
        const float2 scale = make_float2(kScoreLog2, kScoreLog2), shift = make_float2(mc, mc);
        float2 sum0 = make_float2(0.f, 0.f), sum1 = make_float2(0.f, 0.f);
        auto weights = [&](const uint32_t* x, int c) {
          uint32_t p[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float2 y = fma2(make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), scale, shift);
            if (e % kPolyEach == 0) {
              y = exp2_poly(y);
            } else {
              y.x = ex2(y.x);
              y.y = ex2(y.y);
            }
            if (e & 1) sum1 = add2(sum1, y); else sum0 = add2(sum0, y);
            p[e] = cvt_bf16x2(y.x, y.y);
          }
          tmem_st16(s_t + (c >> 1), p);       // over S columns that have been read
        };
#pragma unroll 1
        for (int c = 0; c < 128; c += 64) {
          if (c >= seen) {
            uint32_t none[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) none[e] = 0u;
            tmem_ld_wait();
            tmem_st16(s_t + (c >> 1), none);
            tmem_st16(s_t + (c >> 1) + 16, none);
            continue;
          }
          tmem_ld_wait();
          tmem_ld32(s_t + c + 32, u[1]);
          weights(u[0], c);
          tmem_ld_wait();
          if (c + 64 < seen) tmem_ld32(s_t + 64, u[0]);
          weights(u[1], c + 32);
        }
        if (!fresh && __any_sync(0xffffffffu, f != 1.f)) {
          // what O holds so far is for the old maximum (P V of the step before is done: S came after it)
#pragma unroll 1
          for (int k = 0; k < 128; k += 16) {
            uint32_t o[16];
            tmem_ld16(o_t + k, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st16(o_t + k, o);
          }
        }
        sum0 = add2(sum0, sum1);
        l += sum0.x + sum0.y;
        tmem_st_wait();
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(p_bar);
      ++own_steps;
      fresh = false;
    }
    if (!ok) break;
    // the maximum and the sum, for the output (which has taken the last ones)
    if (own_items > 0 && !pa_wait(smem_u32(&sm.ml_free[slot]), (own_items - 1) & 1, abort_flag, status)) break;
    ++own_items;
    sm.ml[slot][row] = make_float2(m, l);
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sm.ml_full[slot]));
  }
}

// Warps 12-15: the output, a thread for each row.  O is read as soon as its last product is done, and
// given back for the next item's; the softmax is then already at that one.
__device__ __forceinline__ void pa_output(const PromptArgs& a, PaShared& sm, uint32_t tmem) {
  const int warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
  uint32_t* const status = reinterpret_cast<uint32_t*>(a.work);
  volatile int* const abort_flag = &sm.abort_flag;
  const uint32_t o_t = tmem + 256 + (static_cast<uint32_t>(warp) << 21);
  const int row = warp * 32 + lane;
  const int row_tok = row / a.group, row_head = row - row_tok * a.group;
  uint32_t items0 = 0, items1 = 0, single_steps = 0;   // items with steps in slots 0 and 1
  for (uint32_t count = 0;; ++count) {
    if (!pa_item_wait(sm, count, status)) return;
    const PaItem item = sm.items[count % kPaItems];
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sm.item_empty[count % kPaItems]));
    if (item.tokens == 0) return;
    const bool two = item.flags & kPaTwo;
    const int tiles = item.j1 - item.j0;
    const bool has0 = two ? item.end0 > item.j0 : (single_steps & 1) == 0 || tiles > 1;
    const bool has1 = two ? true : (single_steps & 1) == 1 || tiles > 1;
    if (!two) single_steps += tiles;
    const uint32_t phase0 = items0 & 1, phase1 = items1 & 1;
    items0 += has0;
    items1 += has1;
    if (!(item.flags & kPaWhole) && (item.flags & kPaEnds) && threadIdx.x == kPaThreads - 128) {
      // the item's last piece is here: what the joining kernel has to know
      PaJoin* const join = reinterpret_cast<PaJoin*>(a.work + a.off_desc) + static_cast<int>(blockIdx.x);
      join->first = item.first_cta;
      join->tok = item.tok;
      join->tokens = item.tokens;
      join->g = item.g;
      join->valid = 1;
    }
    // a row tile for each slot, or one row tile from both slots
    for (int x = 0; x < (two ? 2 : 1); ++x) {
      const bool use0 = has0 && x == 0, use1 = has1 && (x == 1 || !two);
      float2 ml0 = make_float2(-INFINITY, 0.f), ml1 = ml0;
      if (use0) {
        if (!pa_wait(smem_u32(&sm.ml_full[0]), phase0, abort_flag, status)) return;
        ml0 = sm.ml[0][row];
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.ml_free[0]));
      }
      if (use1) {
        if (!pa_wait(smem_u32(&sm.ml_full[1]), phase1, abort_flag, status)) return;
        ml1 = sm.ml[1][row];
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.ml_free[1]));
      }
      const float m = max3_nan(ml0.x, ml1.x, ml1.x);
      float f0 = ml0.x == -INFINITY ? 0.f : ex2((ml0.x - m) * kScoreLog2);
      float f1 = ml1.x == -INFINITY ? 0.f : ex2((ml1.x - m) * kScoreLog2);
      const float l = ml0.y * f0 + ml1.y * f1;
      const int tok_in_item = x * a.tpt + row_tok;
      const bool live = row_tok < a.tpt && tok_in_item < item.tokens;
      const bool warp_live = __any_sync(0xffffffffu, live);
      const int64_t tok = item.tok + tok_in_item;
      const int head = item.g * a.group + row_head;
      const bool whole = item.flags & kPaWhole;
      const bool direct = whole && a.mode != kPaPrefixOnce;
      float* dst = nullptr;
      uint16_t* quad[4];                                              // the rows of this lane's quad
      uint32_t quad_live = 0;
      if (direct) {
        const float inv = l > 0.f ? 1.f / l : 0.f;
        f0 *= inv;
        f1 *= inv;
        const int64_t off = tok * a.ld_out + static_cast<int64_t>(head) * kHeadDim;
#pragma unroll
        for (int e = 0; e < 4; ++e) quad[e] = a.out + __shfl_sync(0xffffffffu, off, (lane & ~3) + e) + (lane & 3) * 8;
        quad_live = (__ballot_sync(0xffffffffu, live) >> (lane & ~3)) & 15u;
      } else {
        float2* ml;
        if (!whole) {                                                 // a piece: columns in blocks of 4
          const int64_t tile = (static_cast<int64_t>(static_cast<int>(blockIdx.x)) * 2 + (item.flags & kPaCarried ? 0 : 1)) * 2 + x;
          ml = reinterpret_cast<float2*>(a.work + a.off_ml) + tile * 128 + row;
          dst = reinterpret_cast<float*>(a.work + a.off_o) + tile * 128 * kHeadDim + row * 4;
        } else {
          const int64_t r = (item.flags & kPaOnce ? 0 : static_cast<int64_t>(a.n_tok) * a.h_q) + tok * a.h_q + head;
          ml = reinterpret_cast<float2*>(a.work + a.off_row_ml) + r;
          dst = reinterpret_cast<float*>(a.work + a.off_row_o) + r * kHeadDim;
        }
        if (live) *ml = make_float2(m, l);
      }
      if (use0 && !pa_wait(smem_u32(&sm.pv_done[0]), phase0, abort_flag, status)) return;
      if (use1 && !pa_wait(smem_u32(&sm.pv_done[1]), phase1, abort_flag, status)) return;
      tc_fence_after();
      if (warp_live && (use0 || use1)) {
        const int stride = whole ? 4 : 128 * 4;
#pragma unroll 1
        for (int c = 0; c < kHeadDim; c += 32) {
          float r[32];
          if (use0 && use1) {
            uint32_t o[32], u[32];
            tmem_ld32(o_t + c, o);
            tmem_ld32(o_t + 128 + c, u);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) r[e] = fmaf(__uint_as_float(o[e]), f0, __uint_as_float(u[e]) * f1);
          } else {
            uint32_t o[32];
            tmem_ld32(o_t + (use0 ? 0 : 128) + c, o);
            tmem_ld_wait();
            const float f = use0 ? f0 : f1;
#pragma unroll
            for (int e = 0; e < 32; ++e) r[e] = __uint_as_float(o[e]) * f;
          }
          if (direct) {
            // a lane has 64 bytes of its row; after the exchange a quad writes them for one row after another
            uint32_t u[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) u[e] = cvt_bf16x2(r[2 * e], r[2 * e + 1]);
            transpose_quad(u);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if ((quad_live >> e) & 1)
                *reinterpret_cast<uint4*>(quad[e] + c) = make_uint4(u[4 * e], u[4 * e + 1], u[4 * e + 2], u[4 * e + 3]);
          } else if (live) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              *reinterpret_cast<float4*>(dst + (c / 4 + e) * stride) =
                  make_float4(r[4 * e], r[4 * e + 1], r[4 * e + 2], r[4 * e + 3]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (use0) mbar_arrive(smem_u32(&sm.o_free[0]));
        if (use1) mbar_arrive(smem_u32(&sm.o_free[1]));
      }
    }
  }
}

// Warp 11: what is refused is reported, its rows zero.
__device__ __forceinline__ void pa_refuse(const PromptArgs& a, const PaShared& sm) {
  const int lane = threadIdx.x & 31;
  uint32_t* const status = reinterpret_cast<uint32_t*>(a.work);
  const bool all = sm.share.refused, no_prefix = pa_prefix(a) < 0;
  if (static_cast<int>(blockIdx.x) == 0 && lane == 0) {
    reinterpret_cast<PaJoin*>(a.work + a.off_desc)->refused = all;
    if (all || no_prefix) atomicOr(status, kDevBadInput);
  }
  // a sequence at a time; a row, where all are refused
  for (int b = static_cast<int>(blockIdx.x); b < (all ? a.n_tok : a.batch); b += gridDim.x) {
    int64_t t0 = b, t1 = t0 + 1;
    if (!all) {
      const PaSequence s = pa_sequence(a, b);
      if (!s.bad && !no_prefix) continue;
      if (s.bad && lane == 0) atomicOr(status, kDevBadInput);
      t0 = s.tok0 < 0 ? 0 : s.tok0;
      t1 = a.cu ? a.cu[b + 1] : t0 + a.t_new;
      if (t1 > a.n_tok) t1 = a.n_tok;
    }
    const int cols = a.h_q * (kHeadDim / 8);
    for (int64_t t = t0; t < t1; ++t)
      for (int e = lane; e < cols; e += 32)
        *reinterpret_cast<uint4*>(a.out + t * a.ld_out + e * 8) = make_uint4(0, 0, 0, 0);
  }
}

// ---------------------------------------------------------------- the kernel
__global__ void __launch_bounds__(kPaThreads, 1)
    prompt_attention_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                            const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_pk,
                            const __grid_constant__ CUtensorMap tm_pv, const __grid_constant__ PromptArgs a) {
  extern __shared__ __align__(1024) uint8_t pa_dyn[];
  PaShared& sm = *reinterpret_cast<PaShared*>(pa_dyn + kPaTilesBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t q_s = smem_u32(pa_dyn), kv_s = q_s + 2 * kPaTileBytes;
  if (q_s & 1023u) {                     // the swizzled tiles count on it
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (tid == 0) {
      atomicOr(reinterpret_cast<uint32_t*>(a.work), kDevStopped);
      (reinterpret_cast<PaJoin*>(a.work + a.off_desc) + static_cast<int>(blockIdx.x))->valid = 0;
    }
    return;
  }

  if (warp == 8) {
    // the barriers lie one after another: a lane initialises one, or two
    auto count_of = [](int k) -> uint32_t {
      constexpr int kQ = 2 * kPaStages;        // kv_full, kv_empty; q_full, q_empty, s_ready: one arrival
      if (k < kQ + 6) return 1u;
      if (k < kQ + 8) return 4u;               // p_ready
      if (k < kQ + 10) return 1u;              // pv_done
      if (k < kQ + 16) return 4u;              // o_free, ml_full, ml_free
      if (k < kQ + 17 + kPaItems) return 1u;   // drained, item_full
      return 14u;                              // item_empty: loads, products, 8 warps of softmax, 4 of output
    };
    static_assert(offsetof(PaShared, items) == 8 * kPaBarriers && kPaBarriers == 2 * kPaStages + 17 + 2 * kPaItems);
    for (int k = lane; k < kPaBarriers; k += 32)
      mbar_init(smem_u32(&sm.kv_full[0]) + 8 * k, count_of(k) + (k == 0 ? a.test_stall : 0u));
    if (lane == 0) sm.abort_flag = 0;
    __syncwarp();
    if (lane == 0) fence_barrier_init();
    if (lane == 1) prefetch_tensormap(&tm_q);
    if (lane == 2) prefetch_tensormap(&tm_k);
    if (lane == 3) prefetch_tensormap(&tm_v);
    if (lane == 4) prefetch_tensormap(&tm_pk);
    if (lane == 5) prefetch_tensormap(&tm_pv);
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(&sm.tmem), 512);
    tmem_relinquish();
  }
  // Nothing of this call is read or written before the kernels ahead of it are done.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0) (reinterpret_cast<PaJoin*>(a.work + a.off_desc) + static_cast<int>(blockIdx.x))->valid = 0;
  tc_fence_before();
  if (a.batch > kPaWarpBatch) {
    __syncthreads();
    pa_find_share(a, sm);
  } else if (warp != 10) {
    __syncthreads();                     // warp 10 comes to it when it has its first item
  }
  tc_fence_after();
  const uint32_t tmem = sm.tmem;

  // Registers: 512 x 128 at launch = 256 x 160 + 256 x 96, so that a thread of
  // the softmax holds its row of S.
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 160;");
    pa_softmax(a, sm, tmem);
  } else if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
    pa_output(a, sm, tmem);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
    if (warp == 8) pa_load(a, sm, q_s, kv_s, &tm_q, &tm_k, &tm_v, &tm_pk, &tm_pv);
    if (warp == 9) pa_multiply(a, sm, tmem, q_s, kv_s);
    if (warp == 10) pa_find_items(a, sm);
    if (warp == 11) pa_refuse(a, sm);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- joining pieces
// A row's pieces (m, l, O) in order: out = sum e^(m_p - M) O_p / sum e^(m_p - M) l_p.  Bound by the
// latency of L2: all maxima of a row are loaded at once, then all of its O.
__device__ __forceinline__ int64_t pa_piece_tile(int cta, int first, int x) {
  return (static_cast<int64_t>(cta) * 2 + (cta == first ? 1 : 0)) * 2 + x;
}
// The weight of a piece under the maximum of all; 0 for one that has seen nothing (its O is not taken).
__device__ __forceinline__ float pa_piece_weight(float m, float top) {
  return m == -INFINITY ? 0.f : ex2((m - top) * kScoreLog2);
}

// Split items: grid (CTAs of the attention, 8), 8 warps.  A block takes 32 rows, a lane for each (as they
// lie in the pieces), a warp 16 columns.
__global__ void __launch_bounds__(256) prompt_join_kernel(const PromptArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const PaJoin j = reinterpret_cast<const PaJoin*>(a.work + a.off_desc)[blockIdx.x];
  if (!j.valid) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int x = blockIdx.y >> 2, last = blockIdx.x;
  const int row = (blockIdx.y & 3) * 32 + lane;
  const int t = row / a.group;
  if (t >= a.tpt || x * a.tpt + t >= j.tokens) return;
  const float2* const ml = reinterpret_cast<const float2*>(a.work + a.off_ml) + row;
  const float* const o = reinterpret_cast<const float*>(a.work + a.off_o) + (warp * 4 * 128 + row) * 4;
  float m = -INFINITY, l = 0.f;
  float4 acc[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int p = j.first; p <= last; p += 2) {       // almost always there are two
    float2 s[2];
    float4 v[2][4];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int64_t tile = pa_piece_tile(min(p + e, last), j.first, x);
      s[e] = ml[tile * 128];
      if (p + e > last) s[e] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[e][k] = *reinterpret_cast<const float4*>(o + tile * 128 * kHeadDim + k * 128 * 4);
    }
    const float top = max3(m, s[0].x, s[1].x);
    const float f = pa_piece_weight(m, top);
    l *= f;
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] = make_float4(acc[k].x * f, acc[k].y * f, acc[k].z * f, acc[k].w * f);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float w = pa_piece_weight(s[e].x, top);
      l = fmaf(s[e].y, w, l);
      if (w != 0.f) {                  // (NaN too)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          acc[k].x = fmaf(v[e][k].x, w, acc[k].x);
          acc[k].y = fmaf(v[e][k].y, w, acc[k].y);
          acc[k].z = fmaf(v[e][k].z, w, acc[k].z);
          acc[k].w = fmaf(v[e][k].w, w, acc[k].w);
        }
      }
    }
    m = top;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  uint16_t* const dst = a.out + static_cast<int64_t>(j.tok + x * a.tpt + t) * a.ld_out +
                        static_cast<int64_t>(j.g * a.group + row - t * a.group) * kHeadDim + warp * 16;
#pragma unroll
  for (int k = 0; k < 4; k += 2)
    *reinterpret_cast<uint4*>(dst + k * 4) =
        make_uint4(cvt_bf16x2(acc[k].x * inv, acc[k].y * inv), cvt_bf16x2(acc[k].z * inv, acc[k].w * inv),
                   cvt_bf16x2(acc[k + 1].x * inv, acc[k + 1].y * inv), cvt_bf16x2(acc[k + 1].z * inv, acc[k + 1].w * inv));
}

// Every row behind a prefix taken once: its prefix's pieces, then its own keys'.  A warp a row: a lane
// looks after one piece (of 32), then after four columns.
__global__ void __launch_bounds__(256) prefix_join_kernel(const PromptArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t r = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int64_t rows = static_cast<int64_t>(a.n_tok) * a.h_q;
  if (r >= rows) return;
  const int tok = static_cast<int>(div_u64(r, a.h_q)), head = static_cast<int>(r - static_cast<int64_t>(tok) * a.h_q);
  const int g = head / a.group;
  const int prefix = pa_prefix(a);
  int b;
  if (a.cu) {
    if (reinterpret_cast<const PaJoin*>(a.work + a.off_desc)->refused) return;
    if (tok >= a.cu[a.batch] || tok < a.cu[0]) return;
    b = find_sequence(a.cu, a.batch, tok);
  } else {
    b = tok / a.t_new;
  }
  const PaSequence seq = pa_sequence(a, b);
  const int t = tok - seq.tok0;
  if (seq.bad || t < 0 || t >= seq.n || prefix < 0) return;        // what is refused is zero already
  // the CTAs that have the pieces of the prefix's item, and of the own one
  const int2* const owners = reinterpret_cast<const int2*>(a.work + a.off_owners);
  const int in0 = tok % (2 * a.tpt), in1 = t < 2 * a.tpt ? t : t % (2 * a.tpt);     // the token's place in its item
  const int2 c0 = prefix > 0 ? owners[static_cast<int64_t>(tok - in0) * a.h_kv + g] : make_int2(0, -1);
  const int2 c1 = owners[static_cast<int64_t>(a.n_tok) * a.h_kv + static_cast<int64_t>(tok - in1) * a.h_kv + g];
  // (what a call that gave up has left out is not followed)
  auto sound = [&](int2 c) { return c.x >= 0 && c.x <= c.y && c.y < a.ctas; };
  if ((prefix > 0 && !sound(c0)) || !sound(c1)) return;
  const int n0 = c0.y - c0.x + 1, n = n0 + c1.y - c1.x + 1;
  const int in_group = head - g * a.group;
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int p0 = 0; p0 < n; p0 += 32) {
    float2 s = make_float2(-INFINITY, 0.f);
    int64_t at = 0;                                    // where its O is, in 4 floats; whole rows: ~(where)
    if (p0 + lane < n) {
      const bool own = p0 + lane >= n0;
      const int2 c = own ? c1 : c0;
      if (c.x == c.y) {
        const int64_t row = own ? rows + r : r;
        s = reinterpret_cast<const float2*>(a.work + a.off_row_ml)[row];
        at = ~(row * 32);
      } else {
        const int in = own ? in1 : in0, x = in >= a.tpt ? 1 : 0, row = (in - x * a.tpt) * a.group + in_group;
        const int64_t tile = pa_piece_tile(c.x + p0 + lane - (own ? n0 : 0), c.x, x);
        s = reinterpret_cast<const float2*>(a.work + a.off_ml)[tile * 128 + row];
        at = tile * 4096 + row;
      }
    }
    float top = fmaxf(m, s.x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    const float f = pa_piece_weight(m, top);
    const float w = pa_piece_weight(s.x, top);
    float sum = s.y * w;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    l = l * f + sum;
    acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
    m = top;
    const int here = min(32, n - p0);
#pragma unroll 1
    for (int q0 = 0; q0 < here; q0 += 4) {
      float4 v[4];
      float wq[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int q = min(q0 + e, here - 1);
        wq[e] = __shfl_sync(0xffffffffu, w, q);
        if (q0 + e >= here) wq[e] = 0.f;
        const int64_t qa = __shfl_sync(0xffffffffu, at, q);
        const float4* src = qa < 0 ? reinterpret_cast<const float4*>(a.work + a.off_row_o) + ~qa + lane
                                   : reinterpret_cast<const float4*>(a.work + a.off_o) + qa + lane * 128;
        v[e] = *src;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (wq[e] != 0.f) {                            // (NaN too)
          acc.x = fmaf(v[e].x, wq[e], acc.x);
          acc.y = fmaf(v[e].y, wq[e], acc.y);
          acc.z = fmaf(v[e].z, wq[e], acc.z);
          acc.w = fmaf(v[e].w, wq[e], acc.w);
        }
      }
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  *reinterpret_cast<uint2*>(a.out + static_cast<int64_t>(tok) * a.ld_out + static_cast<int64_t>(head) * kHeadDim + lane * 4) =
      make_uint2(cvt_bf16x2(acc.x * inv, acc.y * inv), cvt_bf16x2(acc.z * inv, acc.w * inv));
}

}  // namespace qspec
