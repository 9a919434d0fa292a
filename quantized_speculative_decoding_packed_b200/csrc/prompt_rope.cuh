// Positions of the prompt path: the fused QKV projection's query and key
// heads get their optional per-head norms and their rotation, and the keys
// and values go into the shared cache, in one pass over the projection.
//
// For head row x (128 columns), position p and rotated width R:
//   x <- x / sqrt(mean(x^2) + eps) * gamma               (where a gamma is given)
//   (x_i, x_k) <- (x_i cos a - x_k sin a, x_k cos a + x_i sin a),  a = angle of pair i at p,
// pairs (i, i + R/2), or (2i, 2i + 1) with kRopeInterleaved; columns R..127 pass.
//
// Bound by memory: 4 bytes read and 2 (bf16) or 4 (fp32 queries) written per
// column.  A warp owns a head row (a lane holds 4 consecutive columns, one
// 512-byte load per row), so the norm is one shuffle reduction and the
// partner column of a split pair comes from another lane at the same
// place within its four; up to kRopeHeads rows of a warp are in flight.
// 4900 tokens of 80 heads (302 MB): 58 us, 5.2 TB/s; with
// a resident grid that goes through the tokens 85-90 (its warps wait for the
// small loads in turn, where new CTAs have them under way).
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "attention.cuh"
#include "device_common.cuh"

namespace qspec {

constexpr int kRopeWarps = 4;
constexpr int kRopeHeads = 4;                 // head rows of a warp, loaded together
constexpr int kRopeHeadsPerCta = kRopeWarps * kRopeHeads;

// Two fp32 values rounded to bf16 (nearest even), `lo` in the low half.
__device__ __forceinline__ uint32_t cvt_bf16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

struct RopeArgs {
  const float* qkv;            // no restrict: q_out may be the same rows
  const int32_t* cu;           // null: t_new tokens for every sequence
  const int32_t* lens;
  const int32_t* prefix_len;   // null: 0
  const float* q_gamma;
  const float* k_gamma;
  const float* table;          // [table_rows][rot]: cosines, then sines
  uint16_t* k_cache;
  uint16_t* v_cache;
  void* q_out;
  uint32_t* status;
  int64_t ld, ld_q, table_rows;
  float eps;
  int n_tok, batch, t_new, offset, h_q, h_kv, rot, l_max, interleaved, q_f32;
};

// The sequence of packed token `tok`: the last b with cu[b] <= tok, so that a
// sequence without tokens is passed over.  A warp narrows [0, batch) by a
// factor of 32 in each step.  Always in [0, batch).
__device__ __forceinline__ int find_sequence(const int32_t* __restrict__ cu, int batch, int tok) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = batch;                       // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int at = lo + lane * step;
    const bool le = lane * step < n && (lane == 0 || cu[at] <= tok);
    const int k = 31 - __clz(__ballot_sync(0xffffffffu, le));
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

// grid (tokens, ceil((h_q + 2 h_kv) / kRopeHeadsPerCta)); with starts and a status word one column of CTAs
// more, which looks at the starts (beside the loads of each token's own CTA the same test costs 2 us of 57).
__global__ void __launch_bounds__(kRopeWarps * 32) qkv_rope_append_kernel(const RopeArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tok = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (tok >= a.n_tok) {
    for (int e = threadIdx.x; e < a.batch && blockIdx.y == 0; e += kRopeWarps * 32) {
      const int start = a.cu[e], end = a.cu[e + 1];
      if (start < 0 || start > end || end > a.n_tok || (e == 0 && start != 0)) atomicOr(a.status, kDevBadInput);
    }
    return;
  }
  const int heads = a.h_q + 2 * a.h_kv;
  const float* row = a.qkv + static_cast<int64_t>(tok) * a.ld + lane * 4;
  const int h0 = blockIdx.y * kRopeHeadsPerCta + warp;
  // the rows first: what follows is a chain of small loads
  float x[kRopeHeads][4];
#pragma unroll
  for (int u = 0; u < kRopeHeads; ++u) {
    const int h = h0 + u * kRopeWarps;
    if (h < heads) {
      const float4 v = __ldcs(reinterpret_cast<const float4*>(row + h * kHeadDim));
      x[u][0] = v.x; x[u][1] = v.y; x[u][2] = v.z; x[u][3] = v.w;
    }
  }
  const int64_t pre = a.prefix_len ? *a.prefix_len : 0;
  int b, t;
  int64_t len;
  if (a.cu) {
    // (rows behind the last sequence, and tokens of one whose starts do not fit, are in none)
    int start;
    if (a.batch <= 31) {
      // all starts and lengths at once, a lane each
      const int mine = lane <= a.batch ? a.cu[lane] : -1;
      const int cached = lane < a.batch ? a.lens[lane] : 0;
      const int end = __shfl_down_sync(0xffffffffu, mine, 1);
      const uint32_t in = __ballot_sync(0xffffffffu, static_cast<uint32_t>(mine) <= static_cast<uint32_t>(tok) &&
                                                             tok < end && end <= a.n_tok);
      if (in == 0) return;
      b = 31 - __clz(in);
      start = __shfl_sync(0xffffffffu, mine, b);
      len = __shfl_sync(0xffffffffu, cached, b);
    } else {
      if (tok >= a.cu[a.batch]) return;
      b = find_sequence(a.cu, a.batch, tok);
      start = a.cu[b];
      const int end = a.cu[b + 1];
      len = a.lens[b];
      if (start < 0 || tok < start || tok >= end || end > a.n_tok) return;
    }
    t = tok - start;
  } else {
    b = tok / a.t_new;
    t = tok - b * a.t_new;
    len = a.lens[b];
  }
  const int64_t pos = len + a.offset + t;
  if (len < 0 || pos >= a.l_max || pre < 0 || (a.rot > 0 && pre + pos >= a.table_rows)) {
    if (a.status && threadIdx.x == 0 && blockIdx.y == 0) atomicOr(a.status, kDevBadInput);
    return;
  }
  // this lane's angles: columns 4 lane .. 4 lane + 3
  const int half = a.rot >> 1;
  const bool turned = lane * 4 < a.rot;
  float cs[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
  int partner = lane;
  if (turned) {
    const float* angle = a.table + (pre + pos) * a.rot;
    if (a.interleaved) {
      const float2 c = *reinterpret_cast<const float2*>(angle + lane * 2);
      const float2 s = *reinterpret_cast<const float2*>(angle + half + lane * 2);
      cs[0] = cs[1] = c.x; cs[2] = cs[3] = c.y;
      sn[0] = sn[1] = s.x; sn[2] = sn[3] = s.y;
    } else {
      const int quarter = half >> 2;           // lanes per half (R is a multiple of 8)
      const bool upper = lane >= quarter;
      partner = upper ? lane - quarter : lane + quarter;
      const int i = (upper ? lane - quarter : lane) * 4;
      const float4 c = *reinterpret_cast<const float4*>(angle + i);
      const float4 s = *reinterpret_cast<const float4*>(angle + half + i);
      cs[0] = c.x; cs[1] = c.y; cs[2] = c.z; cs[3] = c.w;
      const float sg = upper ? 1.f : -1.f;
      sn[0] = sg * s.x; sn[1] = sg * s.y; sn[2] = sg * s.z; sn[3] = sg * s.w;
    }
  }
  const int64_t q_at = static_cast<int64_t>(tok) * a.ld_q + lane * 4;
  const int64_t kv_at = (static_cast<int64_t>(b) * a.h_kv * a.l_max + pos) * kHeadDim + lane * 4;
#pragma unroll
  for (int u = 0; u < kRopeHeads; ++u) {
    const int h = h0 + u * kRopeWarps;
    if (h >= heads) break;                     // the same for the whole warp
    const bool is_v = h >= a.h_q + a.h_kv;
    if (!is_v) {
      const float* gamma = h < a.h_q ? a.q_gamma : a.k_gamma;
      if (gamma) {
        float ss = x[u][0] * x[u][0] + x[u][1] * x[u][1] + x[u][2] * x[u][2] + x[u][3] * x[u][3];
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
        const float r = rsqrtf(ss * (1.f / kHeadDim) + a.eps);
        const float4 g = *reinterpret_cast<const float4*>(gamma + lane * 4);
        x[u][0] *= r * g.x; x[u][1] *= r * g.y; x[u][2] *= r * g.z; x[u][3] *= r * g.w;
      }
      if (a.rot > 0) {
        if (a.interleaved) {
          if (turned) {
            const float e0 = x[u][0], e2 = x[u][2];
            x[u][0] = e0 * cs[0] - x[u][1] * sn[0];
            x[u][1] = x[u][1] * cs[1] + e0 * sn[1];
            x[u][2] = e2 * cs[2] - x[u][3] * sn[2];
            x[u][3] = x[u][3] * cs[3] + e2 * sn[3];
          }
        } else {
          float y[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] = __shfl_sync(0xffffffffu, x[u][i], partner);
          if (turned) {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[u][i] = x[u][i] * cs[i] + y[i] * sn[i];
          }
        }
      }
    }
    if (h < a.h_q) {
      if (a.q_f32)
        *reinterpret_cast<float4*>(static_cast<float*>(a.q_out) + q_at + h * kHeadDim) = make_float4(x[u][0], x[u][1], x[u][2], x[u][3]);
      else
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.q_out) + q_at + h * kHeadDim) =
            make_uint2(cvt_bf16x2(x[u][0], x[u][1]), cvt_bf16x2(x[u][2], x[u][3]));
    } else {
      const int g = h - a.h_q - (is_v ? a.h_kv : 0);
      uint16_t* cache = is_v ? a.v_cache : a.k_cache;
      *reinterpret_cast<uint2*>(cache + kv_at + static_cast<int64_t>(g) * a.l_max * kHeadDim) =
          make_uint2(cvt_bf16x2(x[u][0], x[u][1]), cvt_bf16x2(x[u][2], x[u][3]));
    }
  }
}

// table[p][i] = cos(p f_i), table[p][R/2 + i] = sin(p f_i): 64 bits for the
// angle and its functions (at position 10^5 a 32-bit angle is off by 4e-3),
// rounded once.
__global__ void __launch_bounds__(256) rope_table_kernel(const double* __restrict__ inv_freq, int64_t rows,
                                                         int half, float* __restrict__ table) {
  const int64_t e = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (e >= rows * half) return;
  const int64_t p = e / half;
  const int i = static_cast<int>(e - p * half);
  double s, c;
  sincos(static_cast<double>(p) * inv_freq[i], &s, &c);
  table[p * 2 * half + i] = static_cast<float>(c);
  table[p * 2 * half + half + i] = static_cast<float>(s);
}

}  // namespace qspec
