// What the attention kernels share: element conversion, the visibility rule
// and score of cb.h in the form the kernels evaluate it, and the row-by-row
// form that repairs a row whose tiled sum met a hidden infinity or NaN.
//
// Scores are kept in units of log2: x = log2(e) * s, so that exp(s - max)
// is one hardware base-2 exponential.  A query's visible keys are those of
// [0, hi) that share its document, with
//   hi = min(kv_len, causal ? max(i + q_offset + 1, prefix_len) : Lk).
#pragma once

#include <cuda_bf16.h>

#include "internal.h"

namespace cb {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kNegInf = -__builtin_huge_valf();

// Packed pairs of fp32 (fma.rn.f32x2: each lane an fmaf): half the issue slots.
using f2 = unsigned long long;
__device__ __forceinline__ f2 pack2(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(f2 v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Keys of sequence b that exist, and those all its queries see.
struct SeqRule {
  int kv;      // kv_len clamped to [0, Lk]
  int prefix;  // prefix_len clamped to [0, Lk]
};
__device__ __forceinline__ SeqRule seq_rule(const AttnArgs& a, int b) {
  SeqRule r{a.Lk, 0};
  if (a.kv_len) r.kv = min(max(a.kv_len[b], 0), a.Lk);
  if (a.prefix_len) r.prefix = min(max(a.prefix_len[b], 0), a.Lk);
  return r;
}
// End of the keys that query i sees (before documents); grows with i.
__device__ __forceinline__ int row_end(const AttnArgs& a, const SeqRule& r, int i) {
  return a.causal ? max(0, min(r.kv, max(i + a.q_offset + 1, r.prefix))) : r.kv;
}

// log2(e) * score of a dot product; dist = |i + q_offset - j|.
__device__ __forceinline__ float score_log2(const AttnArgs& a, float dot, float slope_log2, int dist) {
  float x = dot * a.scale;
  if (a.softcap > 0.f) x = a.softcap * tanhf(x / a.softcap);
  return fmaf(-slope_log2, static_cast<float>(dist), x * kLog2e);
}

// A row of n elements in 16-byte pieces (VEC) or one by one.
template <typename T>
__device__ __forceinline__ void unpack16(uint4 w, float (&f)[16 / sizeof(T)]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) f[i] = __uint_as_float(u[i]);
    else f[2 * i] = __uint_as_float(u[i] << 16), f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
template <typename T, bool VEC>
__device__ __forceinline__ float row_dot(const T* q, const T* k, int n) {
  float dot = 0.f;
  if constexpr (VEC) {
    constexpr int kPer = 16 / sizeof(T);
#pragma unroll 4
    for (int d = 0; d < n; d += kPer) {
      float x[kPer], y[kPer];
      unpack16<T>(*reinterpret_cast<const uint4*>(q + d), x);
      unpack16<T>(*reinterpret_cast<const uint4*>(k + d), y);
#pragma unroll
      for (int e = 0; e < kPer; ++e) dot = fmaf(x[e], y[e], dot);
    }
  } else {
    for (int d = 0; d < n; ++d) dot = fmaf(to_f32(q[d]), to_f32(k[d]), dot);
  }
  return dot;
}
template <typename T, bool VEC>
__device__ __forceinline__ bool row_finite(const T* v, int n) {
  float zero = 0.f;  // NaN once an element was infinite or NaN
  if constexpr (VEC) {
    constexpr int kPer = 16 / sizeof(T);
#pragma unroll 4
    for (int d = 0; d < n; d += kPer) {
      float x[kPer];
      unpack16<T>(*reinterpret_cast<const uint4*>(v + d), x);
#pragma unroll
      for (int e = 0; e < kPer; ++e) zero = fmaf(x[e], 0.f, zero);
    }
  } else {
    for (int d = 0; d < n; ++d) zero = fmaf(to_f32(v[d]), 0.f, zero);
  }
  return zero == 0.f;
}

// The tiled kernels multiply a masked key's weight 0 into its value, which is
// NaN where that value is infinite or NaN. A row whose result is not finite is
// therefore done again by attn_row, unless the result is what the definition
// gives in any case:
//  - its sum of weights is NaN: a visible score is NaN or +infinity, and a
//    masked one never enters the sum, so every value of the row is NaN;
//  - a value that it sees is not finite, and none that it does not see.
// (Done again for one NaN in a key that every query sees, all rows would take
// seconds over long sequences, and bounded waits behind them would run out.)
// If all values are finite, or the sum is large, weights relative to an early
// maximum may have overflowed: again.
//
// By a whole warp, a row per lane: bad, its result is not finite; hi, doc, the
// keys that it sees; sum, of its weights. end: the keys that its tile
// multiplied, or more. Returns the lanes whose rows are to be done again.
// (A call, as attn_row is: the hot paths keep their registers.)
template <typename T, bool VEC>
__device__ __noinline__ unsigned rows_to_redo(const AttnArgs& a, int b, int hk, int end, bool bad, int hi, int doc, float sum) {
  bad = bad && sum == sum;
  if (!__any_sync(~0u, bad)) return 0;
  const int lane = threadIdx.x & 31;
  const T* v = static_cast<const T*>(a.v) + b * a.vs_b + hk * a.vs_h;
  const int* doc_k = a.doc_k ? a.doc_k + static_cast<long long>(b) * a.Lk : nullptr;
  unsigned seen_bad = 0, hidden_bad = 0;
  for (int j0 = 0; j0 < end; j0 += 32) {
    const int j = j0 + lane;
    const unsigned odd = __ballot_sync(~0u, j < end && !row_finite<T, VEC>(v + j * a.vs_l, a.dv));
    const int n = min(max(hi - j0, 0), 32);
    unsigned seen = n == 32 ? ~0u : (1u << n) - 1;
    if (doc_k)
      for (unsigned x = odd; x; x &= x - 1) {
        const int key = __ffs(x) - 1;
        if (doc_k[j0 + key] != doc) seen &= ~(1u << key);
      }
    seen_bad |= odd & seen;
    hidden_bad |= odd & ~seen;
  }
  return __ballot_sync(~0u, bad && (hidden_bad || !seen_bad || sum > 0x1p24f));
}

// One query row by one warp, key by key, in fp32. A key that is not visible is
// never touched, so the row comes out as defined: finite where the visible
// data is, and infinite or NaN where that is. Values of its result that are
// finite stand: only the others are written.
template <typename T, bool VEC>
__device__ __noinline__ void attn_row(const AttnArgs& a, int b, int h, int i) {
  const int lane = threadIdx.x & 31;
  const T* q = static_cast<const T*>(a.q) + b * a.qs_b + static_cast<long long>(i) * a.qs_l + h * a.qs_h;
  const T* k = static_cast<const T*>(a.k) + b * a.ks_b + (h / a.group) * a.ks_h;
  const T* v = static_cast<const T*>(a.v) + b * a.vs_b + (h / a.group) * a.vs_h;
  T* o = static_cast<T*>(a.o) + b * a.os_b + static_cast<long long>(i) * a.os_l + h * a.os_h;
  const SeqRule rule = seq_rule(a, b);
  const int hi = row_end(a, rule, i);
  const float slope = a.slopes ? a.slopes[h] * kLog2e : 0.f;
  const int* doc_k = a.doc_k ? a.doc_k + static_cast<long long>(b) * a.Lk : nullptr;
  const int doc = a.doc_q ? a.doc_q[static_cast<long long>(b) * a.Lq + i] : 0;
  float m = kNegInf, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int j0 = 0; j0 < hi; j0 += 32) {
    const int j = j0 + lane;
    const bool vis = j < hi && doc >= 0 && (!doc_k || doc_k[j] == doc);
    const unsigned live = __ballot_sync(~0u, vis);
    if (!live) continue;
    const float x = vis ? score_log2(a, row_dot<T, VEC>(q, k + j * a.ks_l, a.dk), slope, abs(i + a.q_offset - j)) : kNegInf;
    float mx = x;
    for (int s = 16; s; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, s));
    const float mn = fmaxf(m, mx), mu = mn == kNegInf ? 0.f : mn;
    const float corr = exp2_approx(m - mu);
    const float p = vis ? exp2_approx(x - mu) : 0.f;
    m = mn;
    l = l * corr + p;
    for (int c = 0; c < 4; ++c) acc[c] *= corr;
    for (int s0 = 0; s0 < 32; s0 += 8) {  // the values of eight keys in flight
      float w[8][4];
#pragma unroll
      for (int u = 0; u < 8; ++u)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          w[u][c] = (live >> (s0 + u)) & 1 && lane + 32 * c < a.dv ? to_f32(v[(j0 + s0 + u) * a.vs_l + lane + 32 * c]) : 0.f;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float ps = __shfl_sync(~0u, p, s0 + u);
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if ((live >> (s0 + u)) & 1) acc[c] = fmaf(ps, w[u][c], acc[c]);
      }
    }
  }
  for (int s = 16; s; s >>= 1) l += __shfl_xor_sync(~0u, l, s);
  __syncwarp();  // the row's result, by whichever lanes, is there to be read
  for (int c = 0; c < 4; ++c)
    if (lane + 32 * c < a.dv && !(to_f32(o[lane + 32 * c]) * 0.f == 0.f)) o[lane + 32 * c] = from_f32<T>(l == 0.f ? 0.f : acc[c] / l);
}

}  // namespace cb
