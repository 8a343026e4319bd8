// What the attention kernels share: element conversion, the visibility rule
// and score of cb.h in the form the kernels evaluate it, and the row-by-row
// form that repairs a row whose tiled sum met an infinity or NaN.
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

// One query row by one warp, key by key, in fp32.  The tiled kernels multiply
// a masked key's weight 0 into its value, which is NaN where that value is
// infinite or NaN; they call this for each row whose result is not finite.
// Here a key that is not visible is never touched, so the row comes out as
// defined: finite where the visible data is, and infinite or NaN where that is.
template <typename T>
__device__ __forceinline__ void attn_row_inline(const AttnArgs& a, int b, int h, int i) {
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
    float x = kNegInf;
    if (vis) {
      float dot = 0.f;
      for (int d = 0; d < a.dk; ++d) dot = fmaf(to_f32(q[d]), to_f32(k[j * a.ks_l + d]), dot);
      x = score_log2(a, dot, slope, abs(i + a.q_offset - j));
    }
    float mx = x;
    for (int s = 16; s; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, s));
    const float mn = fmaxf(m, mx), mu = mn == kNegInf ? 0.f : mn;
    const float corr = exp2_approx(m - mu);
    const float p = vis ? exp2_approx(x - mu) : 0.f;
    m = mn;
    l = l * corr + p;
    for (int c = 0; c < 4; ++c) acc[c] *= corr;
    unsigned live = __ballot_sync(~0u, vis);
    while (live) {
      const int s = __ffs(live) - 1;
      live &= live - 1;
      const float ps = __shfl_sync(~0u, p, s);
      const T* row = v + static_cast<long long>(j0 + s) * a.vs_l;
      for (int c = 0; c < 4; ++c)
        if (lane + 32 * c < a.dv) acc[c] = fmaf(ps, to_f32(row[lane + 32 * c]), acc[c]);
    }
  }
  for (int s = 16; s; s >>= 1) l += __shfl_xor_sync(~0u, l, s);
  for (int c = 0; c < 4; ++c)
    if (lane + 32 * c < a.dv) o[lane + 32 * c] = from_f32<T>(l == 0.f ? 0.f : acc[c] / l);
}

// The same as a call, for kernels whose registers the cold path would burden.
template <typename T>
__device__ __noinline__ void attn_row(const AttnArgs& a, int b, int h, int i) {
  attn_row_inline<T>(a, b, h, i);
}

}  // namespace cb
