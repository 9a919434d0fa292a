// Attention of many new tokens over the shared KV cache: packed causal
// prompts, and batches whose sequences share one prefix.
//
//   out_r = sum_j w_j v_j,  w = softmax_j(q_r . k_j / sqrt(128)) over the keys j that row r sees.
//
// One pass over the keys: for each tile of 128 keys S = Q K^T on the tensor
// cores, the running maximum m and sum l of the softmax in fp32 registers,
// P = exp(S - m) rounded to bf16 (its only rounding; the values are bf16, and
// both operands of the product have one type), O += P V in fp32 tensor
// memory, out = O / l.  m is only raised, and O scaled, when a tile exceeds it
// by more than 2^kRaise: until then P is at most 2^kRaise, with the same
// relative rounding.
//
// A CTA per SM works through its share of the items (prompt_schedule.cuh).
//   warp 8: TMA of queries (ring of two tiles) and of key and value tiles
//           (ring of 5 x 32 KB);
//   warp 9: tcgen05.mma: S of the next step before P V of the current one;
//   warps 0-3, 4-7: the softmax of slots 0 and 1, a thread for each row.  A slot
//           is a tile of S, and of O, in tensor memory; P takes S's place.
// With two row tiles, each has a slot, and both use every key tile.  With one,
// the slots take alternate key tiles and are joined at the end of the item.
// A piece of a split item is left in the workspace as (m, l, O); a second
// kernel joins the pieces in order.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "attention.cuh"
#include "device_common.cuh"
#include "prompt_rope.cuh"
#include "prompt_schedule.cuh"

namespace qspec {

constexpr int kPaStages = 5;
constexpr int kPaThreads = 384;
constexpr int kPaTileBytes = 128 * kHeadDim * 2;             // 32 KB: a tile of Q, K or V
constexpr float kScoreLog2 = kInvSqrtHeadDim * 1.4426950408889634f;   // scores in powers of two
constexpr float kRaise = 8.f;

struct PromptArgs {
  const int32_t* cu;           // null: t_new tokens for every sequence
  const int32_t* lens;
  const int32_t* prefix_len;   // null: no prefix
  uint16_t* out;
  uint8_t* work;
  int64_t ld_out;
  int64_t off_start, off_desc, off_ml, off_o, off_row_ml, off_row_o;
  int n_tok, batch, t_new, offset, h_q, h_kv, group, tpt, l_max, prefix_max;
};

// A split item that ends in a CTA's share: its pieces are those of CTAs first .. this one.
struct PaJoin {
  int32_t valid, first, tok0, n_tok, g, pad[3];
};

struct PaMeta {
  int64_t total;
  int32_t ctas;
  int32_t prefix;              // the prefix's length, -1 where it is refused
};

// Workspace: status word, what the GEMMs keep there, then per CTA two pieces of two row tiles;
// with a prefix, for each (token, head) a row for its prefix and one for its own keys.
constexpr int64_t kPaOffMeta = 8192;
struct PaLayout {
  int64_t off_start, off_desc, off_ml, off_o, off_row_ml, off_row_o, total;
};
__host__ __device__ inline PaLayout pa_layout(int64_t grid, int64_t batch, int64_t rows, bool prefix) {
  PaLayout l;
  auto up = [](int64_t v) { return (v + 255) / 256 * 256; };
  l.off_desc = kPaOffMeta + 256;
  l.off_ml = up(l.off_desc + grid * static_cast<int64_t>(sizeof(PaJoin)));
  l.off_o = up(l.off_ml + grid * 4 * 128 * 8);
  l.off_start = up(l.off_o + grid * 4 * 128 * kHeadDim * 4);
  l.off_row_ml = up(l.off_start + (prefix ? batch * 8 : 0));
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

// A warp's bounded wait without a call: around a call the 128 scores of a row would have to be saved.
__device__ __forceinline__ bool pa_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, uint32_t* status) {
  uint64_t start = 0;
  bool ok = true;
  while (!mbar_try_wait(bar, parity)) {
    const uint64_t now = global_timer_ns();
    if (start == 0) start = now;
    if (*abort_flag || now - start > kWaitLimitNs) {
      if (!*abort_flag) atomicOr(status, kDevTimeout);
      *abort_flag = 1;
      ok = false;
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

// ---------------------------------------------------------------- walking the items
// Sequence b's packed tokens and the keys before them; n = 0 where its
// offsets or its length are not those of the cache.
struct PaSequence {
  int tok0, n;
  int64_t base;
  bool bad;
};
__device__ __forceinline__ PaSequence pa_sequence(const PromptArgs& a, int b) {
  PaSequence s;
  int n;
  s.bad = false;
  if (a.cu) {
    s.tok0 = a.cu[b];
    const int64_t end = a.cu[b + 1];
    s.bad = s.tok0 < 0 || end < s.tok0 || end > a.n_tok;
    n = s.bad ? 0 : static_cast<int>(end - s.tok0);
  } else {
    s.tok0 = b * a.t_new;
    n = a.t_new;
  }
  const int64_t len = a.lens[b];
  s.base = len + a.offset;
  s.bad = s.bad || len < 0 || s.base + n > a.l_max;
  s.n = s.bad ? 0 : n;
  return s;
}

// The tokens that take part in the prefix's items.
__device__ __forceinline__ int pa_packed_tokens(const PromptArgs& a) {
  if (!a.cu) return a.n_tok;
  const int end = a.cu[a.batch];
  return end < 0 ? 0 : (end > a.n_tok ? a.n_tok : end);
}

struct PaShare {
  int64_t s0, s1, total;
  int64_t start;               // of the first item
  int b, g, i;                 // the first item; b < 0: the prefix's
  int ctas, prefix;
};

struct PaWalk {
  int64_t start;
  Run run;
  int b, g, i, items, tok0;
  // the item at hand
  int w, n, j0, j1, tokens;

  __device__ __forceinline__ void load_run(const PromptArgs& a, int prefix) {
    run.tpt = a.tpt;
    if (b < 0) {
      run.n = pa_packed_tokens(a);
      run.base = -1;
      run.keys = prefix;
      tok0 = 0;
    } else {
      const PaSequence s = pa_sequence(a, b);
      run.n = s.n;
      run.base = s.base;
      run.keys = 0;
      tok0 = s.tok0;
    }
    items = run_items(run);
  }
  __device__ __forceinline__ void item(const PaShare& sh) {
    tokens = item_tokens(run, i);
    w = tokens > run.tpt ? 2 : 1;
    n = static_cast<int>((item_keys(run, i, tokens) + 127) / 128);
    share_tiles(start, w, n, sh.s0, sh.s1, &j0, &j1);
  }
  __device__ __forceinline__ void begin(const PromptArgs& a, const PaShare& sh) {
    b = sh.b; g = sh.g; i = sh.i; start = sh.start;
    load_run(a, sh.prefix);
  }
  // Moves to the next item with key tiles in the share; false where there is none.
  __device__ __forceinline__ bool find(const PromptArgs& a, const PaShare& sh, bool first) {
    for (;;) {
      if (!first) {
        start += static_cast<int64_t>(w) * n + kItemCost;
        if (++i >= items) {
          i = 0;
          if (++g >= a.h_kv) {
            g = 0;
            do {
              if (++b >= a.batch) return false;
              load_run(a, sh.prefix);
            } while (run.n == 0);
          }
        }
      }
      first = false;
      if (start >= sh.s1) return false;
      item(sh);
      if (j0 < j1) return true;
    }
  }
  // Key tiles of the first row tile in this share end here (the second sees more).
  __device__ __forceinline__ int end_of_first() const {
    if (w == 1 || run.base < 0) return j1;
    const int n0 = static_cast<int>((item_keys(run, i, run.tpt) + 127) / 128);
    return n0 < j1 ? (n0 > j0 ? n0 : j0) : j1;
  }
  __device__ __forceinline__ int64_t last_keys() const { return item_keys(run, i, tokens); }
};

// Barriers and small exchanges in shared memory.
struct PaShared {
  uint64_t kv_full[kPaStages], kv_empty[kPaStages], q_full[2], q_empty[2];
  uint64_t s_ready[2], p_ready[2], pv_done[2], o_free, ml_ready, drained;
  PaShare share;
  int64_t warp_sums[kPaThreads / 32];
  int64_t found_start, found_cost;
  int found_b;
  int abort_flag;
  uint32_t tmem;
  float2 ml[2][128];
};
constexpr int kPaTilesBytes = (2 + kPaStages) * kPaTileBytes;          // Q, K and V tiles, then PaShared
constexpr int kPaSmemBytes = kPaTilesBytes + static_cast<int>(sizeof(PaShared));
static_assert(kPaSmemBytes <= 227 * 1024, "shared memory of a CTA");

// The costs of all sequences, their sum, and this CTA's first item.
__device__ __forceinline__ void pa_find_share(const PromptArgs& a, PaShared& sm) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int prefix = 0;
  if (a.prefix_len) {
    prefix = *a.prefix_len;
    if (prefix < 0 || prefix > a.prefix_max) prefix = 0;
  }
  Run pr;
  pr.n = prefix > 0 ? pa_packed_tokens(a) : 0;
  pr.tpt = a.tpt;
  pr.base = -1;
  pr.keys = prefix;
  const int64_t prefix_head = run_cost(pr);
  const int64_t prefix_all = prefix_head * a.h_kv;

  int64_t before = prefix_all;         // the cost before the chunk of sequences at hand
  int64_t cost = 0, at = 0;
  auto scan = [&](int b) {             // block-wide: this thread's cost and the costs before it
    cost = 0;
    if (b < a.batch) {
      const PaSequence s = pa_sequence(a, b);
      Run r;
      r.n = s.n;
      r.tpt = a.tpt;
      r.base = s.base;
      r.keys = 0;
      cost = run_cost(r) * a.h_kv;
    }
    int64_t incl = cost;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t o = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += o;
    }
    if (lane == 31) sm.warp_sums[warp] = incl;
    __syncthreads();
    int64_t all = 0;
    at = before + incl - cost;
#pragma unroll
    for (int k = 0; k < kPaThreads / 32; ++k) {
      const int64_t s = sm.warp_sums[k];
      if (k < warp) at += s;
      all += s;
    }
    before += all;
    __syncthreads();
  };
  for (int b0 = 0; b0 < a.batch; b0 += kPaThreads) scan(b0 + tid);
  const int64_t total = before;
  const int ctas = working_ctas(total, gridDim.x);
  const int c = blockIdx.x;
  const int64_t s0 = c < ctas ? share_start(total, ctas, c) : total;
  const int64_t s1 = c < ctas ? share_start(total, ctas, c + 1) : total;
  if (tid == 0) {
    sm.share.s0 = s0;
    sm.share.s1 = s1;
    sm.share.total = total;
    sm.share.ctas = ctas;
    sm.share.prefix = prefix;
    sm.found_b = -1;
  }
  if (c == 0 && tid == 0) {
    PaMeta* meta = reinterpret_cast<PaMeta*>(a.work + kPaOffMeta);
    meta->total = total;
    meta->ctas = ctas;
    meta->prefix = a.prefix_len && *a.prefix_len != prefix ? -1 : prefix;
  }
  __syncthreads();
  int64_t* const starts = a.prefix_len ? reinterpret_cast<int64_t*>(a.work + a.off_start) : nullptr;
  before = prefix_all;
  for (int b0 = 0; b0 < a.batch; b0 += kPaThreads) {
    const int b = b0 + tid;
    if (a.batch > kPaThreads) scan(b);           // else this thread's values still stand
    if (b < a.batch) {
      if (c == 0 && starts) starts[b] = at;
      if (cost > 0 && at <= s0 && s0 < at + cost) {
        sm.found_b = b;
        sm.found_start = at;
        sm.found_cost = cost / a.h_kv;
      }
    }
  }
  __syncthreads();
  if (s0 < s1 && warp == 0) {
    int b = sm.found_b, g;
    int64_t start, head_cost;
    Run r;
    if (s0 < prefix_all) {
      b = -1;
      start = 0;
      head_cost = prefix_head;
      r = pr;
    } else {
      start = sm.found_start;
      head_cost = sm.found_cost;
      const PaSequence s = pa_sequence(a, b);
      r.n = s.n;
      r.tpt = a.tpt;
      r.base = s.base;
      r.keys = 0;
    }
    g = static_cast<int>((s0 - start) / head_cost);
    start += g * head_cost;
    // the last item that starts at or before s0: [lo, lo + n) narrowed 32-fold
    int lo = 0, n = run_items(r);
    while (n > 1) {
      const int step = (n + 31) / 32;
      const bool le = lane * step < n && (lane == 0 || start + cost_before(r, lo + lane * step) <= s0);
      const int k = 31 - __clz(__ballot_sync(0xffffffffu, le));
      lo += k * step;
      n = min(step, n - k * step);
    }
    if (lane == 0) {
      sm.share.b = b;
      sm.share.g = g;
      sm.share.i = lo;
      sm.share.start = start + cost_before(r, lo);
    }
  }
  __syncthreads();
}

// ---------------------------------------------------------------- the softmax of one tile
// Row of S in tensor memory -> P (bf16) in its place; m, l updated.  Returns
// the factor by which what is in O has to be scaled (1: nothing to do).
struct PaRow {
  float m;                     // the maximum in use (-inf: none yet)
  float l;
};

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
// Two fp32 values rounded to bf16 (nearest even), `lo` in the low half.
__device__ __forceinline__ uint32_t cvt_bf16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// ---------------------------------------------------------------- the roles of the warps
__device__ __forceinline__ void pa_load(const PromptArgs& a, PaShared& sm, uint32_t q_s, uint32_t kv_s,
                                        const CUtensorMap* tm_q, const CUtensorMap* tm_k, const CUtensorMap* tm_v,
                                        const CUtensorMap* tm_pk, const CUtensorMap* tm_pv) {
  const int lane = threadIdx.x & 31;
  const PaShare& sh = sm.share;
  uint32_t* const status = reinterpret_cast<uint32_t*>(a.work);
  volatile int* const abort_flag = &sm.abort_flag;
  if (lane == 0) {
    uint32_t ring = 0, qn = 0;
    bool ok = true;
    PaWalk it;
    it.begin(a, sh);
    for (bool first = true; ok && it.find(a, sh, first); first = false) {
      const CUtensorMap* mk = it.b < 0 ? tm_pk : tm_k;
      const CUtensorMap* mv = it.b < 0 ? tm_pv : tm_v;
      const int head = it.b < 0 ? it.g : it.b * a.h_kv + it.g;
      // (a first row tile that sees none of the share's keys is left out)
      for (int x = it.w == 2 && it.end_of_first() == it.j0; x < it.w && ok; ++x, ++qn) {
        const uint32_t slot = qn & 1;
        ok = mbar_wait(smem_u32(&sm.q_empty[slot]), ((qn >> 1) & 1) ^ 1, abort_flag, status);
        if (!ok) break;
        const uint32_t bar = smem_u32(&sm.q_full[slot]);
        const uint32_t dst = q_s + slot * kPaTileBytes;
        mbar_arrive_expect_tx(bar, static_cast<uint32_t>(a.tpt * a.group) * kHeadDim * 2);
        const int tok = it.tok0 + (it.i * 2 + x) * a.tpt;
        tma_load_3d(dst, tm_q, bar, 0, it.g * a.group, tok);
        tma_load_3d(dst + kPaTileBytes / 2, tm_q, bar, 64, it.g * a.group, tok);
      }
      for (int j = it.j0; j < it.j1 && ok; ++j) {
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const uint32_t st = ring % kPaStages;
          ok = ok && mbar_wait(smem_u32(&sm.kv_empty[st]), ((ring / kPaStages) & 1) ^ 1, abort_flag, status);
          if (!ok) break;
          const uint32_t bar = smem_u32(&sm.kv_full[st]);
          mbar_arrive_expect_tx(bar, kPaTileBytes);
          tma_load_4d(kv_s + st * kPaTileBytes, kv ? mv : mk, bar, 0, j * 128, 0, head);
          ++ring;
        }
      }
    }
    if (!ok) {
      // given up: let the copies in flight land before shared memory goes
      const uint32_t kv_from = ring > kPaStages ? ring - kPaStages : 0;
      for (uint32_t r = kv_from; r < ring; ++r)
        mbar_wait_drain(smem_u32(&sm.kv_full[r % kPaStages]), (r / kPaStages) & 1);
      for (uint32_t r = qn > 2 ? qn - 2 : 0; r < qn; ++r)
        mbar_wait_drain(smem_u32(&sm.q_full[r & 1]), (r >> 1) & 1);
    }
  }
  __syncwarp();
}

__device__ __forceinline__ void pa_multiply(const PromptArgs& a, PaShared& sm, uint32_t tmem, uint32_t q_s, uint32_t kv_s) {
  const int lane = threadIdx.x & 31;
  const PaShare& sh = sm.share;
  uint32_t* const status = reinterpret_cast<uint32_t*>(a.work);
  volatile int* const abort_flag = &sm.abort_flag;
  // The steps of the share in order: (row tile or alternate slot, key tile).
  // S of the next step is issued before P V of the current one where its
  // operands are there and its slot is another.
  struct Step {
    uint32_t slot, k_ring, q_ring;     // the value tile is the next in the ring
    int pv_steps, tail;                // 16-key steps of P V; first unseen key of the tile (128: none)
    bool first, fresh;                 // first of its slot in the item, first of the item
    bool k_last, q_last;               // the last step on this key tile, on these queries
  };
  PaWalk it;
  it.begin(a, sh);
  bool have = it.find(a, sh, true);
  int j = 0, x = 0, end0 = 0;
  int64_t last = 0;
  uint32_t ring = 0, qn = 0, count = 0;      // key tiles x 2, query tiles, single-tile steps
  uint32_t item_parity = 0;
  bool entered = false;
  auto next = [&](Step& s) -> bool {
    if (!have) return false;
    bool fresh = false;
    if (!entered) {
      entered = true;
      fresh = true;
      j = it.j0;
      end0 = it.end_of_first();
      last = it.last_keys();
      x = 0;
      item_parity = count & 1;
    }
    const bool two = it.w == 2;
    if (two && x == 0 && j >= end0) x = 1;
    s.fresh = fresh;
    if (two) {
      s.slot = x;
      s.q_ring = qn + (x == 1 && end0 > it.j0);
      s.first = j == it.j0;
      s.k_last = x == 1;
      s.q_last = x == 0 ? j == end0 - 1 : j == it.j1 - 1;
    } else {
      s.slot = (item_parity + (j - it.j0)) & 1;
      s.q_ring = qn;
      s.first = j - it.j0 < 2;
      s.k_last = true;
      s.q_last = j == it.j1 - 1;
    }
    s.k_ring = ring;
    const int64_t left = last - static_cast<int64_t>(j) * 128;
    s.tail = left >= 128 ? 128 : static_cast<int>(left);
    s.pv_steps = (s.tail + 15) / 16;
    // advance
    if (two && x == 0) {
      x = 1;
    } else {
      x = 0;
      ring += 2;
      if (++j >= it.j1) {
        if (!two) count += it.j1 - it.j0;
        qn += two && end0 > it.j0 ? 2 : 1;
        entered = false;
        have = it.find(a, sh, false);
      }
    }
    return true;
  };
  uint32_t p_count = 0;                      // phases of p_ready: slot 0 in bit 0, slot 1 in bit 1
  uint32_t items_done = 0;
  bool ok = true;
  const uint32_t leader = elect_one_lane();
  auto s_operands = [&](const Step& s, bool block) -> bool {
    const uint32_t kb = smem_u32(&sm.kv_full[s.k_ring % kPaStages]), kp = (s.k_ring / kPaStages) & 1;
    const uint32_t qb = smem_u32(&sm.q_full[s.q_ring & 1]), qp = (s.q_ring >> 1) & 1;
    if (!block)
      return __all_sync(0xffffffffu, mbar_test_wait(qb, qp) && mbar_test_wait(kb, kp));
    return warp_wait(qb, qp, abort_flag, status) && warp_wait(kb, kp, abort_flag, status);
  };
  auto issue_s = [&](const Step& s) {
    tc_fence_after();
    if (leader) {
      const uint32_t qa = q_s + (s.q_ring & 1) * kPaTileBytes;
      const uint32_t ka = kv_s + (s.k_ring % kPaStages) * kPaTileBytes;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t off = (k >> 2) * (kPaTileBytes / 2) + (k & 3) * 32;
        mma_ss_bf16(tmem + s.slot * 128, smem_desc_sw128(qa + off), smem_desc_sw128(ka + off), kIdescScores,
                    k > 0);
      }
      mma_commit(smem_u32(&sm.s_ready[s.slot]));
      if (s.k_last) mma_commit(smem_u32(&sm.kv_empty[s.k_ring % kPaStages]));
      if (s.q_last) mma_commit(smem_u32(&sm.q_empty[s.q_ring & 1]));
    }
    __syncwarp();
  };
  auto issue_pv = [&](const Step& s) -> bool {
    const uint32_t r = s.k_ring + 1, st = r % kPaStages;
    if (s.fresh) {                    // the item before has read its O
      if (items_done > 0 && !warp_wait(smem_u32(&sm.o_free), (items_done - 1) & 1, abort_flag, status)) return false;
      ++items_done;
    }
    if (!warp_wait(smem_u32(&sm.kv_full[st]), (r / kPaStages) & 1, abort_flag, status)) return false;
    const uint32_t va = kv_s + st * kPaTileBytes;
    if (s.tail & 15) {
      // keys past the last one seen may hold anything: their weights are 0, their values are made 0
      const int rows = s.pv_steps * 16 - s.tail;
      for (int e = lane; e < rows * 16; e += 32) {
        const uint32_t at = va + ((e >> 3) & 1) * (kPaTileBytes / 2) + (s.tail + (e >> 4)) * 128 + (e & 7) * 16;
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0) : "memory");
      }
      fence_proxy_async_smem();
      __syncwarp();
    }
    if (!warp_wait(smem_u32(&sm.p_ready[s.slot]), (p_count >> s.slot) & 1, abort_flag, status)) return false;
    p_count ^= 1u << s.slot;
    tc_fence_after();
    if (leader) {
      for (int k = 0; k < s.pv_steps; ++k)
        mma_ts<false>(tmem + 256 + s.slot * 128, tmem + s.slot * 128 + k * 8, smem_desc_rows_n(va + k * 2048),
                      kIdescValues, !(s.first && k == 0));
      mma_commit(smem_u32(&sm.pv_done[s.slot]));
      if (s.k_last) mma_commit(smem_u32(&sm.kv_empty[st]));
    }
    __syncwarp();
    return true;
  };
  Step cur, nxt;
  bool more = next(cur);
  if (more) {
    ok = s_operands(cur, true);
    if (ok) issue_s(cur);
  }
  while (ok && more) {
    const bool has_next = next(nxt);
    bool issued = false;
    if (has_next && nxt.slot != cur.slot && s_operands(nxt, false)) {
      issue_s(nxt);
      issued = true;
    }
    ok = issue_pv(cur);
    if (ok && has_next && !issued) {
      ok = s_operands(nxt, true);
      if (ok) issue_s(nxt);
    }
    cur = nxt;
    more = has_next;
  }
  if (!ok) {
    // given up: the products in flight end before tensor memory goes
    if (leader) mma_commit(smem_u32(&sm.drained));
    __syncwarp();
    mbar_wait_drain(smem_u32(&sm.drained), 0);
  }
}

__device__ __forceinline__ void pa_softmax(const PromptArgs& a, PaShared& sm, uint32_t tmem, PaJoin* join) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const PaShare& sh = sm.share;
  uint32_t* const status = reinterpret_cast<uint32_t*>(a.work);
  volatile int* const abort_flag = &sm.abort_flag;
  const uint32_t slot = warp >> 2;
  const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;       // lane base of this warp, in bits 16..
  const int row = (warp & 3) * 32 + lane;
  const uint32_t s_t = tmem + slot * 128 + lanes, o_t = tmem + 256 + lanes;
  const int row_tok = row / a.group, row_head = row - row_tok * a.group;
  uint32_t own_steps = 0, other_steps = 0;   // of this slot and the other so far
  uint32_t count = 0, items = 0, singles = 0;
  bool ok = true;
  PaWalk it;
  it.begin(a, sh);
  for (bool first = true; ok && it.find(a, sh, first); first = false) {
    const bool two = it.w == 2;
    const int end0 = it.end_of_first();
    const int x = two ? static_cast<int>(slot) : 0;                   // this thread's row tile
    // this row: its token, and the keys that it sees
    const int tok_in_item = x * a.tpt + row_tok;
    const bool live = row_tok < a.tpt && tok_in_item < it.tokens;
    const int64_t sees = it.run.base < 0 ? it.run.keys
                                         : it.run.base + static_cast<int64_t>(it.i) * 2 * a.tpt + tok_in_item + 1;
    const bool warp_live = __any_sync(0xffffffffu, live);
    const int64_t least = __shfl_sync(0xffffffffu, sees, 0);          // rows see more and more
    const uint32_t par = count & 1;
    int j, step, end;
    if (two) {
      j = it.j0;
      step = 1;
      end = slot == 0 ? end0 : it.j1;
    } else {
      j = it.j0 + ((slot ^ par) & 1);
      step = 2;
      end = it.j1;
      count += it.j1 - it.j0;
    }
    float m = -INFINITY, l = 0.f;
    bool fresh = true;
    for (; j < end; j += step) {
      if (!pa_wait(smem_u32(&sm.s_ready[slot]), own_steps & 1, abort_flag, status)) { ok = false; break; }
      if (warp_live) {
        tc_fence_after();
        float v[128];
#pragma unroll
        for (int k = 0; k < 4; ++k) tmem_ld32(s_t + k * 32, reinterpret_cast<uint32_t*>(v) + k * 32);
        tmem_ld_wait();
        if (static_cast<int64_t>(j) * 128 + 128 > least) {
          const int64_t left = sees - static_cast<int64_t>(j) * 128;
          const int lim = left >= 128 ? 128 : (left < 0 ? 0 : static_cast<int>(left));
#pragma unroll
          for (int k = 0; k < 128; ++k) v[k] = k < lim ? v[k] : -INFINITY;
        }
        float t0 = v[0], t1 = v[1], t2 = v[2], t3 = v[3];
#pragma unroll
        for (int k = 4; k < 128; k += 8) {
          t0 = fmaxf(t0, fmaxf(v[k], v[k + 1]));
          t1 = fmaxf(t1, fmaxf(v[k + 2], v[k + 3]));
          if (k + 4 < 128) {
            t2 = fmaxf(t2, fmaxf(v[k + 4], v[k + 5]));
            t3 = fmaxf(t3, fmaxf(v[k + 6], v[k + 7]));
          }
        }
        const float top = fmaxf(m, fmaxf(fmaxf(t0, t1), fmaxf(t2, t3)));
        const bool raise = (top - m) * kScoreLog2 > kRaise;           // false where both are -inf
        if (__any_sync(0xffffffffu, raise)) {
          const float f = raise ? ex2((m - top) * kScoreLog2) : 1.f;
          l *= f;
          if (raise) m = top;
          if (!fresh) {
            // what O holds so far is for the old maximum
            if (!pa_wait(smem_u32(&sm.pv_done[slot]), (own_steps - 1) & 1, abort_flag, status)) {
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int k = 0; k < 128; k += 16) {
              uint32_t o[16];
              tmem_ld16(o_t + slot * 128 + k, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st16(o_t + slot * 128 + k, o);
            }
          }
        }
        const float mc = m == -INFINITY ? 0.f : -m * kScoreLog2;
        const float2 scale = make_float2(kScoreLog2, kScoreLog2), shift = make_float2(mc, mc);
        float2 sum0 = make_float2(0.f, 0.f), sum1 = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t p[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float2 y = fma2(make_float2(v[k * 32 + 2 * e], v[k * 32 + 2 * e + 1]), scale, shift);
            y.x = ex2(y.x);
            y.y = ex2(y.y);
            if (e & 1) sum1 = add2(sum1, y); else sum0 = add2(sum0, y);
            p[e] = cvt_bf16x2(y.x, y.y);
          }
          tmem_st16(s_t + k * 16, p);
        }
        sum0 = add2(sum0, sum1);
        l += sum0.x + sum0.y;
        tmem_st_wait();
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.p_ready[slot]));
      ++own_steps;
      fresh = false;
    }
    if (!ok) break;
    const bool whole = it.j0 == 0 && it.j1 == it.n;
    const bool carried = it.start < sh.s0;                            // the item began in an earlier share
    // ---- output: a row tile for each slot, or both slots' halves of one
    float f_own = 1.f, f_other = 0.f;
    bool has_own = true, has_other = false;
    const uint32_t other = slot ^ 1;
    if (two) {
      has_own = end > it.j0;
      other_steps += (slot == 0 ? it.j1 : end0) - it.j0;
    } else {
      const int tiles = it.j1 - it.j0;
      const int mine = (tiles + ((slot ^ par) & 1 ? 0 : 1)) >> 1, theirs = tiles - mine;
      has_own = mine > 0;
      has_other = theirs > 0;
      other_steps += theirs;
      // (the item before has been read: both slots are done with its maxima too)
      if (items > 0 && !pa_wait(smem_u32(&sm.o_free), (items - 1) & 1, abort_flag, status)) { ok = false; break; }
      sm.ml[slot][row] = make_float2(m, l);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.ml_ready));
      if (!pa_wait(smem_u32(&sm.ml_ready), singles & 1, abort_flag, status)) { ok = false; break; }
      ++singles;
      const float2 o = sm.ml[other][row];
      const float top = fmaxf(m, o.x);
      f_own = m == -INFINITY ? 0.f : ex2((m - top) * kScoreLog2);
      f_other = o.x == -INFINITY ? 0.f : ex2((o.x - top) * kScoreLog2);
      l = l * f_own + o.y * f_other;
      m = top;
    }
    if (has_own && !pa_wait(smem_u32(&sm.pv_done[slot]), (own_steps - 1) & 1, abort_flag, status)) { ok = false; break; }
    if (has_other && !pa_wait(smem_u32(&sm.pv_done[other]), (other_steps - 1) & 1, abort_flag, status)) { ok = false; break; }
    tc_fence_after();
    if (warp_live) {
      const int c0 = two ? 0 : static_cast<int>(slot) * 64, c1 = two ? 128 : c0 + 64;
      const int tok = it.tok0 + it.i * 2 * a.tpt + tok_in_item;
      const int head = it.g * a.group + row_head;
      const bool direct = whole && !a.prefix_len;
      const float inv = l > 0.f ? 1.f / l : 0.f;
      const float k_own = direct ? f_own * inv : f_own, k_other = direct ? f_other * inv : f_other;
      float* dst = nullptr;
      if (!direct) {
        float2* ml;
        if (whole) {
          const int64_t r = (it.b < 0 ? 0 : static_cast<int64_t>(a.n_tok) * a.h_q) + static_cast<int64_t>(tok) * a.h_q + head;
          ml = reinterpret_cast<float2*>(a.work + a.off_row_ml) + r;
          dst = reinterpret_cast<float*>(a.work + a.off_row_o) + r * kHeadDim;
        } else {
          const int64_t r = ((static_cast<int64_t>(blockIdx.x) * 2 + (carried ? 0 : 1)) * 2 + x) * 128 + row;
          ml = reinterpret_cast<float2*>(a.work + a.off_ml) + r;
          dst = reinterpret_cast<float*>(a.work + a.off_o) + r * kHeadDim;
        }
        if (live && (two || slot == 0)) *ml = make_float2(m, l);
      }
      uint16_t* const out = a.out + static_cast<int64_t>(tok) * a.ld_out + static_cast<int64_t>(head) * kHeadDim;
#pragma unroll 1
      for (int c = c0; c < c1; c += 32) {
        uint32_t o[32], u[32];
        if (has_own) tmem_ld32(o_t + slot * 128 + c, o);
        if (has_other) tmem_ld32(o_t + other * 128 + c, u);
        tmem_ld_wait();
        float r[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          r[e] = has_own ? __uint_as_float(o[e]) * k_own : 0.f;
          if (has_other) r[e] = fmaf(__uint_as_float(u[e]), k_other, r[e]);
        }
        if (live) {
          if (direct) {
#pragma unroll
            for (int e = 0; e < 32; e += 8)
              *reinterpret_cast<uint4*>(out + c + e) =
                  make_uint4(cvt_bf16x2(r[e], r[e + 1]), cvt_bf16x2(r[e + 2], r[e + 3]),
                             cvt_bf16x2(r[e + 4], r[e + 5]), cvt_bf16x2(r[e + 6], r[e + 7]));
          } else {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<float4*>(dst + c + e) = make_float4(r[e], r[e + 1], r[e + 2], r[e + 3]);
          }
        }
      }
      tc_fence_before();
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sm.o_free));
    ++items;
    if (tid == 0 && !whole && it.j1 == it.n) {
      // the item's last piece is here: what the joining kernel has to know
      join->first = share_owner(sh.total, sh.ctas, it.start);
      join->tok0 = it.tok0 + it.i * 2 * a.tpt;
      join->n_tok = it.tokens;
      join->g = it.g;
      join->valid = 1;
    }
  }
}

// What is refused: reported, its rows zero (warps 10 and 11).
__device__ __forceinline__ void pa_refuse(const PromptArgs& a, PaShared& sm) {
  const int tid = threadIdx.x;
  const PaShare& sh = sm.share;
  uint32_t* const status = reinterpret_cast<uint32_t*>(a.work);
  for (int b = blockIdx.x; b < a.batch; b += gridDim.x) {
    const PaSequence s = pa_sequence(a, b);
    if (!s.bad) continue;
    if (tid == 320) atomicOr(status, kDevBadInput);
    const int64_t t0 = s.tok0 < 0 ? 0 : s.tok0;
    int64_t t1 = a.cu ? a.cu[b + 1] : t0 + a.t_new;
    if (t1 > a.n_tok) t1 = a.n_tok;
    const int cols = a.h_q * (kHeadDim / 8);
    for (int64_t e = tid - 320; e < (t1 - t0) * cols; e += kPaThreads - 320)
      *reinterpret_cast<uint4*>(a.out + (t0 + e / cols) * a.ld_out + (e % cols) * 8) = make_uint4(0, 0, 0, 0);
  }
  if (a.prefix_len && blockIdx.x == 0 && tid == 320 && *a.prefix_len != sh.prefix) atomicOr(status, kDevBadInput);
}

// ---------------------------------------------------------------- the kernel
__global__ void __launch_bounds__(kPaThreads, 1)
    prompt_attention_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                            const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_pk,
                            const __grid_constant__ CUtensorMap tm_pv, const PromptArgs a) {
  extern __shared__ __align__(1024) uint8_t pa_dyn[];
  PaShared& sm = *reinterpret_cast<PaShared*>(pa_dyn + kPaTilesBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t q_s = smem_u32(pa_dyn), kv_s = q_s + 2 * kPaTileBytes;
  uint32_t* const status = reinterpret_cast<uint32_t*>(a.work);
  if (q_s & 1023u) {                     // the swizzled tiles count on it
    if (tid == 0) atomicOr(status, kDevTimeout);
    return;
  }

  if (warp == 8) {
    if (lane == 0) {
      for (int k = 0; k < kPaStages; ++k) {
        mbar_init(smem_u32(&sm.kv_full[k]), 1);
        mbar_init(smem_u32(&sm.kv_empty[k]), 1);
      }
      for (int k = 0; k < 2; ++k) {
        mbar_init(smem_u32(&sm.q_full[k]), 1);
        mbar_init(smem_u32(&sm.q_empty[k]), 1);
        mbar_init(smem_u32(&sm.s_ready[k]), 1);
        mbar_init(smem_u32(&sm.p_ready[k]), 4);
        mbar_init(smem_u32(&sm.pv_done[k]), 1);
      }
      mbar_init(smem_u32(&sm.o_free), 8);
      mbar_init(smem_u32(&sm.ml_ready), 8);
      mbar_init(smem_u32(&sm.drained), 1);
      sm.abort_flag = 0;
      fence_barrier_init();
    }
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
  tc_fence_before();
  pa_find_share(a, sm);
  tc_fence_after();
  const PaShare& sh = sm.share;
  const uint32_t tmem = sm.tmem;
  PaJoin* const join = reinterpret_cast<PaJoin*>(a.work + a.off_desc) + blockIdx.x;
  if (tid == 0) join->valid = 0;

  const bool work = sh.s0 < sh.s1;

  // Registers: 384 x 168 at launch = 256 x 208 + 128 x 88, so that a thread of
  // the softmax holds its row of S.
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    if (work) pa_softmax(a, sm, tmem, join);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp >= 10)
      pa_refuse(a, sm);
    else if (work && warp == 8)
      pa_load(a, sm, q_s, kv_s, &tm_q, &tm_k, &tm_v, &tm_pk, &tm_pv);
    else if (work)
      pa_multiply(a, sm, tmem, q_s, kv_s);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- joining pieces
// A row's pieces (m, l, O) in order: out = sum e^(m_p - M) O_p / sum e^(m_p - M) l_p.
// A warp holds a row, four columns a lane.
struct PaJoined {
  float m, l;
  float4 o;
  __device__ __forceinline__ void add(float2 ml, const float* src, int lane) {
    if (ml.y <= 0.f) return;                     // nothing seen: O is not read
    const float top = fmaxf(m, ml.x);
    const float f = m == -INFINITY ? 0.f : ex2((m - top) * kScoreLog2);
    const float g = ex2((ml.x - top) * kScoreLog2);
    const float4 v = *reinterpret_cast<const float4*>(src + lane * 4);
    o.x = o.x * f + v.x * g;
    o.y = o.y * f + v.y * g;
    o.z = o.z * f + v.z * g;
    o.w = o.w * f + v.w * g;
    l = l * f + ml.y * g;
    m = top;
  }
  __device__ __forceinline__ void pieces(const PromptArgs& a, int first, int last, int x, int row, int lane) {
    for (int c = first; c <= last; ++c) {
      const int64_t r = ((static_cast<int64_t>(c) * 2 + (c == first ? 1 : 0)) * 2 + x) * 128 + row;
      add(reinterpret_cast<const float2*>(a.work + a.off_ml)[r],
          reinterpret_cast<const float*>(a.work + a.off_o) + r * kHeadDim, lane);
    }
  }
  __device__ __forceinline__ void store(const PromptArgs& a, int tok, int head, int lane) const {
    const float inv = l > 0.f ? 1.f / l : 0.f;
    *reinterpret_cast<uint2*>(a.out + static_cast<int64_t>(tok) * a.ld_out + static_cast<int64_t>(head) * kHeadDim +
                              lane * 4) =
        make_uint2(cvt_bf16x2(o.x * inv, o.y * inv), cvt_bf16x2(o.z * inv, o.w * inv));
  }
};

// Split items of packed prompts: grid (CTAs of the attention, 8), 8 warps; a block takes 32 rows.
__global__ void __launch_bounds__(256) prompt_join_kernel(const PromptArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const PaJoin j = reinterpret_cast<const PaJoin*>(a.work + a.off_desc)[blockIdx.x];
  if (!j.valid) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int x = blockIdx.y >> 2;
  for (int k = 0; k < 4; ++k) {
    const int row = (blockIdx.y & 3) * 32 + k * 8 + warp;
    const int t = row / a.group;
    if (t >= a.tpt || x * a.tpt + t >= j.n_tok) return;
    PaJoined s{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    s.pieces(a, j.first, blockIdx.x, x, row, lane);
    s.store(a, j.tok0 + x * a.tpt + t, j.g * a.group + row - t * a.group, lane);
  }
}

// Every row behind a shared prefix: its prefix's pieces, then its own keys'.  A warp a row.
__global__ void __launch_bounds__(256) prefix_join_kernel(const PromptArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t r = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (r >= static_cast<int64_t>(a.n_tok) * a.h_q) return;
  const int tok = static_cast<int>(r / a.h_q), head = static_cast<int>(r - static_cast<int64_t>(tok) * a.h_q);
  const int g = head / a.group;
  int b;
  if (a.cu) {
    if (tok >= a.cu[a.batch] || tok < a.cu[0]) return;
    b = find_sequence(a.cu, a.batch, tok);
  } else {
    b = tok / a.t_new;
  }
  const PaSequence seq = pa_sequence(a, b);
  const int t = tok - seq.tok0;
  if (seq.bad || t < 0 || t >= seq.n) return;            // a refused sequence's rows are zero already
  const PaMeta meta = *reinterpret_cast<const PaMeta*>(a.work + kPaOffMeta);
  PaJoined s{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  auto part = [&](const Run& run, int64_t start, int t, int64_t whole_row) {   // t: the token's place in the run
    const int i = t / (2 * a.tpt), x = (t / a.tpt) & 1;
    start += cost_before(run, i);
    const int w = item_row_tiles(run, i);
    const int n = static_cast<int>((item_keys(run, i, item_tokens(run, i)) + 127) / 128);
    const int first = share_owner(meta.total, meta.ctas, start);
    const int last = share_owner(meta.total, meta.ctas, start + static_cast<int64_t>(w) * (n - 1));
    if (first == last)
      s.add(reinterpret_cast<const float2*>(a.work + a.off_row_ml)[whole_row],
            reinterpret_cast<const float*>(a.work + a.off_row_o) + whole_row * kHeadDim, lane);
    else
      s.pieces(a, first, last, x, (t % a.tpt) * a.group + head - g * a.group, lane);
  };
  Run run;
  run.tpt = a.tpt;
  if (meta.prefix < 0) {                                 // refused: zero
    s.store(a, tok, head, lane);
    return;
  }
  if (meta.prefix > 0) {
    run.n = pa_packed_tokens(a);
    run.base = -1;
    run.keys = meta.prefix;
    part(run, run_cost(run) * g, tok, r);
  }
  run.n = seq.n;
  run.base = seq.base;
  run.keys = 0;
  part(run, reinterpret_cast<const int64_t*>(a.work + a.off_start)[b] + run_cost(run) * g, t,
       static_cast<int64_t>(a.n_tok) * a.h_q + r);
  s.store(a, tok, head, lane);
}

}  // namespace qspec
