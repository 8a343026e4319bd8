// The streaming kernel of attention over a 4-bit cache (cb_attention_decode4),
// for rows of whole 16-byte pieces (dims that are multiples of 32).  Tokens are
// dealt as in decode_common.cuh; a CTA's four warps walk a piece together, each
// its own kStep tokens of every 4 kStep through its own ring of cp.async copies,
// as in decode_stream.cuh.
//
// 4.5 bits an element: at the memory's rate an SM has to turn 42 elements a
// cycle into products, three lane-instructions each.  So codes go to the MMAs
// (m16n8k16, f16 operands, fp32 sums) with one AND and half a shift a pair:
// the bits of a nibble, alone in 16 bits, are the f16 number code * 2^-24, and
// of the nibble above it code * 2^-20; ldmatrix hands each lane whole bytes of a
// token (keys) or of two tokens' same dims (values, transposed).  What is left:
//  - the nibbles hold c + 8.  Keys: 8 sum q of a group goes in as the
//    accumulator's first value.  Values: one more MMA with -8 everywhere per
//    tile, in the same step, so that no sum grows with the offset.
//  - a group's scale: keys, one FMA per score and group on the group's sum;
//    values, on the weights, a set of weights per group.
//  - f16's range.  Queries are scaled by a power of two per head (2^15 above),
//    weights times scales by one per warp, 2^7 below which the largest scale so
//    far lies; O follows when it grows, as it does a maximum.  Weights below
//    2^-31 of the largest are lost.
// The MMAs cut what they add off at the largest term's last bits, toward zero.
// For fp32 that would show, so there queries are two whole numbers of at most
// 2^11 on a common grid per head (hi + lo 2^-12, 24 bits below the largest
// element): every product and sum of theirs is exact.  Weights are sums of two
// f16 numbers (22 bits), and a step's products are added to O by FADDs: cut off
// at O's last bit in every step, they would lose 2^-23 of it each time.
#pragma once

#include <cuda_fp16.h>

#include "cache4.cuh"
#include "decode_stream.cuh"

namespace cb {

__device__ __forceinline__ void cp_async_small(uint32_t dst, const void* src, bool valid, int bytes) {
  if (bytes == 8) asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(valid ? 8 : 0) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(valid ? 4 : 0) : "memory");
}
__device__ __forceinline__ void ldsm4_4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
// d (16 x 8, fp32) += a (16 x 16, f16) * b (16 x 8, f16)
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// What f16 rounding left of a pair: another pair of f16 numbers.
__device__ __forceinline__ uint32_t half2_rest(float lo, float hi, uint32_t bits) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&bits));
  return half2_bits(lo - f.x, hi - f.y);
}

constexpr uint32_t kLowNibble = 0x000f000fu, kHighNibble = 0x00f000f0u;  // times 2^-24, 2^-20
constexpr uint32_t kLowMinus8 = 0x80088008u, kHighMinus8 = 0x80808080u;  // -8 in their units
// Codes as f16 numbers of their own: 1024 + c + 8, then 1024 + 16 (c + 8).
__device__ __forceinline__ uint32_t low_codes(uint32_t w) {
  const uint32_t x = (w & kLowNibble) | 0x64006400u;
  const __half2 h = __hadd2(*reinterpret_cast<const __half2*>(&x), __float2half2_rn(-1032.f));
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t high_codes(uint32_t w) {
  const uint32_t x = (w & kHighNibble) | 0x64006400u;
  const __half2 h = __hfma2(*reinterpret_cast<const __half2*>(&x), __float2half2_rn(0.0625f), __float2half2_rn(-72.f));
  return *reinterpret_cast<const uint32_t*>(&h);
}
constexpr int kWeightBits = 7;  // weights times the largest scale: up to 2^(kDecodeGrowth + kWeightBits) = 2^15
constexpr int kMinTopExp = -119;  // 2^(kWeightBits - top_exp) is an fp32 number

template <int DK_, int DV_, int NB_, typename T_>
struct Decode4Shape {
  using T = T_;
  static constexpr int DK = DK_, DV = DV_, NB = NB_, kStep = 16, kStages = 4, kHeads = 8 * NB_;
  static constexpr int kParts = sizeof(T) == 4 ? 2 : 1;
  static constexpr int GK = DK / kGroup4, GV = DV / kGroup4;
  static constexpr int kKeyBytes = DK / 2, kValBytes = DV / 2;
  static constexpr int kKeyScales = kStep * (kKeyBytes + kValBytes), kValScales = kKeyScales + kStep * GK * 2;  // in a stage
  static constexpr int kStageBytes = kValScales + kStep * GV * 2;
  static constexpr int kRing = kDecodeWarps * kStages * kStageBytes;
  static constexpr int kResults = 4 * (kDecodeWarps + 1) * kHeads * DV;  // the warps' and the CTA's, when a piece ends
  static constexpr int kMain = kRing > kResults ? kRing : kResults;
  static constexpr int kScaleArea = 2 * kStep * 16;  // a step's scales as fp32, per warp
  static constexpr int kSmem = kMain + kDecodeWarps * kScaleArea;
  static constexpr int kCtasPerSm = decode4_ctas_per_sm(DK, DV, sizeof(T) == 2, kHeads, 0);
};

// Row r's 16-byte piece p lies at p ^ swizzle(r): ldmatrix reads one piece of eight rows.
template <int BYTES>
__device__ __forceinline__ constexpr int swizzle4(int row) {
  return BYTES == 64 ? (row >> 1) & 3 : (row >> 2) & 1;
}

template <class S>
struct Decode4Math {
  using T = typename S::T;
  static constexpr int GK = S::GK, GV = S::GV, NB = S::NB;
  DecodeScore score;
  bool bias;
  int g, t4, heads, top_exp;
  uint32_t k_src, v_src;  // this lane's ldmatrix rows
  // Queries as the MMAs' B operand, for each group and its two MMAs: head g, dims 8 t4 + (0, 4) and (1, 5) / 16, then
  // (2, 6) and (3, 7) / 16.
  uint32_t qf[S::kParts][GK][NB][4];
  float first[S::kParts][GK][NB][2];  // -8 sum q of this thread's heads 8 nb + 2 t4 and the one after
  float k_mul, head_mul[NB][2];
  float slope[NB][2], m[NB][2], l[NB][2], o[2 * GV][NB][4];

  __device__ __forceinline__ Decode4Math(const DecodeArgs& a, const Piece& pc) : score(a) {
    const int lane = threadIdx.x & 31;
    g = lane >> 2, t4 = lane & 3, heads = pc.heads, top_exp = kMinTopExp;
    bias = a.slopes != nullptr;
    const int row = (lane & 7) + 8 * ((lane >> 3) & 1);
    k_src = row * S::kKeyBytes + (((lane >> 4) ^ swizzle4<S::kKeyBytes>(row)) * 16);
    v_src = row * S::kValBytes + (((lane >> 4) ^ swizzle4<S::kValBytes>(row)) * 16);
    int exponent[NB], top = -1000;
    float sums[S::kParts][GK][NB];
    constexpr int kBits = S::kParts == 2 ? 11 : 15;  // queries go up to 2^kBits
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int hd = g + 8 * nb;
      const T* q = static_cast<const T*>(a.q) + pc.b * a.qs_b + (pc.h0 + (hd < heads ? hd : 0)) * a.qs_h;
      float x[GK][8], big = 0.f;
#pragma unroll
      for (int i = 0; i < GK; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int d = 32 * i + 8 * t4 + e;
          x[i][e] = hd < heads && d < a.dk ? to_f32(q[d]) : 0.f;
          big = fmaxf(big, fabsf(x[i][e]));
        }
      big = fmaxf(big, __shfl_xor_sync(~0u, big, 1));
      big = fmaxf(big, __shfl_xor_sync(~0u, big, 2));
      int e2 = 0;
      if (big > 0.f && big < __builtin_huge_valf()) frexpf(big, &e2);
      exponent[nb] = e2 - kBits;
      if (big > 0.f) top = max(top, exponent[nb]);
#pragma unroll
      for (int i = 0; i < GK; ++i) {
        float sum[S::kParts] = {};
#pragma unroll
        for (int r = 0; r < 4; ++r) {  // dims 8 t4 + r and r + 4; odd r: a sixteenth
          const float lo = ldexpf(x[i][r], kBits - e2), hi = ldexpf(x[i][r + 4], kBits - e2), unit = r & 1 ? 0.0625f : 1.f;
          if constexpr (S::kParts == 1) {
            qf[0][i][nb][r] = half2_bits(lo * unit, hi * unit);
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&qf[0][i][nb][r]));
            sum[0] += (f.x + f.y) / unit;
          } else {
            const float a0 = rintf(lo), a1 = rintf(hi), b0 = rintf((lo - a0) * 0x1p12f), b1 = rintf((hi - a1) * 0x1p12f);
            qf[0][i][nb][r] = half2_bits(a0 * unit, a1 * unit);
            qf[1][i][nb][r] = half2_bits(b0 * unit, b1 * unit);
            sum[0] += a0 + a1;
            sum[1] += b0 + b1;
          }
        }
#pragma unroll
        for (int p = 0; p < S::kParts; ++p) {
          sum[p] += __shfl_xor_sync(~0u, sum[p], 1);
          sum[p] += __shfl_xor_sync(~0u, sum[p], 2);
          sums[p][i][nb] = sum[p] * (-8.f * 0x1p-24f);
        }
      }
    }
    for (int s = 4; s < 32; s <<= 1) top = max(top, __shfl_xor_sync(~0u, top, s));
    const int k_exp = min(max(top + 24, -126), 127);
    k_mul = ldexpf(1.f, k_exp);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int from = 4 * (2 * t4 + e), hd = 8 * nb + 2 * t4 + e;
        const int he = __shfl_sync(~0u, exponent[nb], from);
        head_mul[nb][e] = ldexpf(1.f, min(he + 24 - k_exp, 16)) * (score.cap ? 1.f : score.c_scale);
#pragma unroll
        for (int p = 0; p < S::kParts; ++p)
#pragma unroll
          for (int i = 0; i < GK; ++i) first[p][i][nb][e] = __shfl_sync(~0u, sums[p][i][nb], from);
        slope[nb][e] = a.slopes && hd < heads ? a.slopes[pc.h0 + hd] * kLog2e : 0.f;
        m[nb][e] = kNegInf;
        l[nb][e] = 0.f;
      }
#pragma unroll
      for (int d = 0; d < 2 * GV; ++d)
#pragma unroll
        for (int r = 0; r < 4; ++r) o[d][nb][r] = 0.f;
    }
  }

  __device__ __forceinline__ void rescale(const float (&f)[NB][2]) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int d = 0; d < 2 * GV; ++d)
#pragma unroll
        for (int r = 0; r < 4; ++r) o[d][nb][r] *= f[nb][r & 1];
  }

  // 16 tokens of a stage; bit x of lv: token x exists; far: the first one's distance from the query.  area: this
  // warp's scales as fp32, [keys, values][token][group].
  __device__ __forceinline__ void step(uint32_t st, unsigned lv, int far, const DecodeArgs& a, float4* area) {
    const int lane = threadIdx.x & 31;
    {  // lanes 0 to 15: the keys' scales of their token; 16 to 31: the values'
      const bool is_v = lane >= 16;
      const int groups = is_v ? GV : GK, real = is_v ? a.dv : a.dk;
      const uint32_t at = st + (is_v ? S::kValScales + (lane - 16) * GV * 2 : S::kKeyScales + lane * GK * 2);
      uint32_t w0, w1 = 0;
      if (GK == GV ? GK == 4 : groups == 4) asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w0), "=r"(w1) : "r"(at) : "memory");
      else asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w0) : "r"(at) : "memory");
      const bool live = (lv >> (lane & 15)) & 1;
      if (!live) w0 = w1 = 0;
      if (real <= 32) w0 &= 0xffffu;
      if (real <= 96) w1 &= 0xffffu;
      float4 f = make_float4(__uint_as_float(w0 << 16), __uint_as_float(w0 & 0xffff0000u), __uint_as_float(w1 << 16),
                             __uint_as_float(w1 & 0xffff0000u));
      float big = is_v ? fmaxf(fmaxf(f.x, f.y), fmaxf(f.z, f.w)) : 0.f;  // NaN only where all are
      if (!(big < __builtin_huge_valf())) big = 0.f;
      const unsigned top = __reduce_max_sync(~0u, __float_as_uint(big));
      const int e = static_cast<int>(top >> 23) - 126;  // below 2^e
      if (e > top_exp) {
        const float f2 = exp2_approx(static_cast<float>(top_exp - e));
        top_exp = e;
        float all[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) all[nb][0] = all[nb][1] = f2;
        rescale(all);
      }
      const float mul = is_v ? __uint_as_float(static_cast<unsigned>(127 + kWeightBits - top_exp) << 23) : k_mul;
      f.x *= mul, f.y *= mul, f.z *= mul, f.w *= mul;
      area[lane] = f;
      __syncwarp();
    }
    float s[NB][4];  // element r: key g + 8 (r >> 1), head 8 nb + 2 t4 + (r & 1)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int r = 0; r < 4; ++r) s[nb][r] = 0.f;
    {
      const float4 x0 = area[g], x1 = area[g + 8];
      const float k0[4] = {x0.x, x0.y, x0.z, x0.w}, k1[4] = {x1.x, x1.y, x1.z, x1.w};
#pragma unroll
      for (int i = 0; i < GK; i += 2) {
        uint32_t w[4];  // groups i and i + 1: a word of key g and of key g + 8
        ldsm4_4((st + k_src) ^ (i * 16), w);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t u = w[2 * j], v = w[2 * j + 1], u8 = u >> 8, v8 = v >> 8;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            float acc[S::kParts][4];
#pragma unroll
            for (int p = 0; p < S::kParts; ++p) {
              const float(&f)[2] = first[p][i + j][nb];
              acc[p][0] = acc[p][2] = f[0], acc[p][1] = acc[p][3] = f[1];
              const uint32_t(&q)[4] = qf[p][i + j][nb];
              mma_f16(acc[p], u & kLowNibble, v & kLowNibble, u & kHighNibble, v & kHighNibble, q[0], q[1]);
              mma_f16(acc[p], u8 & kLowNibble, v8 & kLowNibble, u8 & kHighNibble, v8 & kHighNibble, q[2], q[3]);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float sum = S::kParts == 2 ? fmaf(acc[S::kParts - 1][r], 0x1p-12f, acc[0][r]) : acc[0][r];
              s[nb][r] = fmaf(sum, r < 2 ? k0[i + j] : k1[i + j], s[nb][r]);
            }
          }
        }
      }
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int r = 0; r < 4; ++r) s[nb][r] *= head_mul[nb][r & 1];
    if (score.cap) score(s);  // x = log2(e) * score
    const float dist = static_cast<float>(far - g);
    bool grow = false;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float x = s[nb][r];
        if (bias) x = fmaf(-slope[nb][r & 1], dist - 8.f * (r >> 1), x);
        if (lv != 0xffffu && !((lv >> (g + 8 * (r >> 1))) & 1)) x = kNegInf;
        s[nb][r] = x;
        grow |= x > m[nb][r & 1] + kDecodeGrowth;
      }
    if (__any_sync(~0u, grow)) {
      float f[NB][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float y = fmaxf(s[nb][e], s[nb][2 + e]);
          y = fmaxf(y, __shfl_xor_sync(~0u, y, 4));
          y = fmaxf(y, __shfl_xor_sync(~0u, y, 8));
          y = fmaxf(y, __shfl_xor_sync(~0u, y, 16));
          const float mn = fmaxf(m[nb][e], y);
          f[nb][e] = mn == kNegInf ? 1.f : exp2_approx(m[nb][e] - mn);
          m[nb][e] = mn;
          l[nb][e] *= f[nb][e];
        }
      rescale(f);
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const float mu0 = m[nb][0] == kNegInf ? 0.f : m[nb][0], mu1 = m[nb][1] == kNegInf ? 0.f : m[nb][1];
#pragma unroll
      for (int r = 0; r < 4; ++r) s[nb][r] = exp2_approx(s[nb][r] - (r & 1 ? mu1 : mu0));
      l[nb][0] += s[nb][0] + s[nb][2];
      l[nb][1] += s[nb][1] + s[nb][3];
    }
    const float4 x0 = area[16 + g], x1 = area[24 + g];
    const float v0[4] = {x0.x, x0.y, x0.z, x0.w}, v1[4] = {x1.x, x1.y, x1.z, x1.w};
#pragma unroll
    for (int i = 0; i < GV; i += 2) {
      uint32_t w[4];  // groups i and i + 1: dims 4 g .. + 4 of tokens 2 t4, 2 t4 + 1 and of those + 8
      ldsm4_4t((st + S::kStep * S::kKeyBytes + v_src) ^ (i * 16), w);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t u = w[2 * j], v = w[2 * j + 1], u8 = u >> 8, v8 = v >> 8;
        const float c0 = v0[i + j], c1 = v1[i + j];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const float p0 = s[nb][0] * c0, p1 = s[nb][1] * c0, p2 = s[nb][2] * c1, p3 = s[nb][3] * c1;
          uint32_t lo = half2_bits(p0, p1), hi = half2_bits(p2, p3);
          if constexpr (S::kParts == 1) {
            const uint32_t b0 = transpose8x8(lo), b1 = transpose8x8(hi);
            float(&d0)[4] = o[2 * (i + j)][nb], (&d1)[4] = o[2 * (i + j) + 1][nb];
            mma_f16(d0, u & kLowNibble, u & kHighNibble, v & kLowNibble, v & kHighNibble, b0, b1);
            mma_f16(d1, u8 & kLowNibble, u8 & kHighNibble, v8 & kLowNibble, v8 & kHighNibble, b0, b1);
            mma_f16(d0, kLowMinus8, kHighMinus8, kLowMinus8, kHighMinus8, b0, b1);
            mma_f16(d1, kLowMinus8, kHighMinus8, kLowMinus8, kHighMinus8, b0, b1);
          } else {
            float fresh[2][4] = {};
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              if (p) lo = half2_rest(p0, p1, lo), hi = half2_rest(p2, p3, hi);
              const uint32_t b0 = transpose8x8(lo), b1 = transpose8x8(hi);
              mma_f16(fresh[0], low_codes(u), high_codes(u), low_codes(v), high_codes(v), b0, b1);
              mma_f16(fresh[1], low_codes(u8), high_codes(u8), low_codes(v8), high_codes(v8), b0, b1);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) o[2 * (i + j)][nb][r] += fresh[0][r], o[2 * (i + j) + 1][nb][r] += fresh[1][r];
          }
        }
      }
    }
  }

  // This warp's results: res[heads][DV] divided by their sum of weights (so they are no larger than the values are),
  // the maxima with that sum in them, and sums of 1 (0: no token).
  __device__ __forceinline__ void store(float* res, float* ms, float* ls) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float y = l[nb][e];
        y += __shfl_xor_sync(~0u, y, 4);
        y += __shfl_xor_sync(~0u, y, 8);
        y += __shfl_xor_sync(~0u, y, 16);
        const int hd = 8 * nb + 2 * t4 + e;
        if (g == 0) ms[hd] = y == 0.f ? kNegInf : m[nb][e] + log2f(y), ls[hd] = y == 0.f ? 0.f : y == y ? 1.f : y;
        const float inv = y == 0.f ? 0.f : 1.f / y;
        if (hd < heads)
#pragma unroll
          for (int d = 0; d < 2 * GV; ++d)
            *reinterpret_cast<float2*>(res + hd * S::DV + 16 * (d & ~1) + 4 * g + 2 * (d & 1)) =
                make_float2(ldexpf(o[d][nb][e] * inv, top_exp - kWeightBits + (S::kParts == 1 ? 24 : 0)),
                            ldexpf(o[d][nb][2 + e] * inv, top_exp - kWeightBits + (S::kParts == 1 ? 20 : 0)));
      }
  }
};

template <class S, bool WHOLE>
__global__ void __launch_bounds__(kDecodeThreads, S::kCtasPerSm) decode4_stream_kernel(const DecodeArgs a) {
  using T = typename S::T;
  constexpr int DV = S::DV, kStep = S::kStep, kStages = S::kStages;
  constexpr int CK = S::kKeyBytes / 16, CV = S::kValBytes / 16, RK = 32 / CK, RV = 32 / CV;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float ms[kDecodeWarps][S::kHeads], ls[kDecodeWarps][S::kHeads];
  __shared__ float part_m[S::kHeads], part_l[S::kHeads];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int kq = a.dk / kGroup4, vq = a.dv / kGroup4;  // real pieces per row; what the others hold meets queries of 0
  pdl_wait();
  pdl_launch_dependents();
  const int per_seq = a.Hkv * a.chunks;
  unsigned* prefix = reinterpret_cast<unsigned*>(smem + S::kSmem);
  long long at = 0, end = 1, cta = blockIdx.x;
  Run run{1, 1};
  int b = 0;
  if constexpr (!WHOLE) {
    tile_prefix(a, prefix);
    const long long total = static_cast<long long>(prefix[a.B]) * per_seq;
    run = Run{total, min(static_cast<long long>(gridDim.x), max(total, 1LL))};
    if (tid == 0) a.record[2 * cta] = -1;
    zero_empty(a, prefix, [&](long long i) { static_cast<T*>(a.o)[i] = from_f32<T>(0.f); });
    if (cta >= run.ctas || total == 0) return;
    at = run.begin(cta);
    end = run.begin(cta + 1);
    b = find_seq(a, prefix, per_seq, at);
  }
  const uint32_t ring = smem_u32(smem + warp * kStages * S::kStageBytes);
  float4* area = reinterpret_cast<float4*>(smem + S::kMain + warp * S::kScaleArea);
  const uint32_t k_dst = (lane / CK) * S::kKeyBytes + (((lane % CK) ^ swizzle4<S::kKeyBytes>(lane / CK)) * 16);
  const uint32_t v_dst = kStep * S::kKeyBytes + (lane / CV) * S::kValBytes + (((lane % CV) ^ swizzle4<S::kValBytes>(lane / CV)) * 16);
  const uint32_t x_dst = lane < 16 ? S::kKeyScales + lane * S::GK * 2 : S::kValScales + (lane - 16) * S::GV * 2;
  const long long xs_p = lane < 16 ? a.cache.kx_p : a.cache.vx_p, xs_t = lane < 16 ? a.cache.kx_t : a.cache.vx_t;
  const bool same = a.cache.ks_p == a.cache.vs_p && a.cache.ks_t == a.cache.vs_t;  // one offset serves both
  // from a lane's token to its next one, without a division per step
  const int adv_pg = kDecodeWarps * kStep / a.cache.page_size, adv_slot = kDecodeWarps * kStep - adv_pg * a.cache.page_size;

  while (at < end) {
    Piece pc;
    if constexpr (WHOLE) pc = whole_piece(a, per_seq);
    else pc = next_piece(a, prefix, per_seq, at, end, &b);
    const char* kbase = static_cast<const char*>(a.cache.k) + pc.hk * a.cache.ks_h + (lane % CK) * 16;
    const char* vbase = static_cast<const char*>(a.cache.v) + pc.hk * a.cache.vs_h + (lane % CV) * 16;
    const uint16_t* xbase = lane < 16 ? a.cache.k_scale + pc.hk * a.cache.kx_h : a.cache.v_scale + pc.hk * a.cache.vx_h;

    const int base = pc.tile0 * kDecodeTile + warp * kStep;
    const int steps = pc.tiles * (kDecodeTile / (kDecodeWarps * kStep));
    // Lanes look the step's tokens up (lane and lane + 16 the same one), one step before their copies are issued:
    // the byte offsets of the rows, or -1.
    struct Rows {
      long long k, v, x;
    };
    unsigned j = base + lane % kStep;  // unsigned: a token looked up past the piece's end may be past 2^31
    int pg = static_cast<int>(j) / a.cache.page_size, slot = static_cast<int>(j) - pg * a.cache.page_size;
    auto lookup = [&](int step) {  // once for each step, in order
      Rows r{-1, -1, 0};
      if (step < steps && j >= static_cast<unsigned>(pc.lo) && j < static_cast<unsigned>(pc.hi)) {
        const long long page = checked_page(a, pc.b, pg);
        if (page >= 0) {
          r.k = page * a.cache.ks_p + slot * a.cache.ks_t;
          r.v = same ? r.k : page * a.cache.vs_p + slot * a.cache.vs_t;
          r.x = page * xs_p + slot * xs_t;
        }
      }
      j += kDecodeWarps * kStep;
      pg += adv_pg, slot += adv_slot;
      if (slot >= a.cache.page_size) slot -= a.cache.page_size, ++pg;
      return r;
    };
    unsigned live[kStages];  // bit x: token x of the stage's step exists
    auto issue = [&](int step, int stage, const Rows& rows) {
      const unsigned have = __ballot_sync(~0u, rows.k >= 0) & 0xffffu;
      if (step < steps) {
        const uint32_t st = ring + stage * S::kStageBytes;
#pragma unroll
        for (int i = 0; i < kStep / RK; ++i) {
          const int r = i * RK + lane / CK;
          const long long off = __shfl_sync(~0u, rows.k, r);
          const bool ok = (have >> r) & 1;
          if (lane % CK < kq) cp_async16((st + k_dst + i * RK * S::kKeyBytes) ^ (swizzle4<S::kKeyBytes>(i * RK) * 16), ok ? kbase + off : kbase, ok);
          if (CK == CV) {
            const long long to = same ? off : __shfl_sync(~0u, rows.v, r);
            if (lane % CV < vq) cp_async16((st + v_dst + i * RV * S::kValBytes) ^ (swizzle4<S::kValBytes>(i * RV) * 16), ok ? vbase + to : vbase, ok);
          }
        }
        if (CK != CV) {
#pragma unroll
          for (int i = 0; i < kStep / RV; ++i) {
            const int r = i * RV + lane / CV;
            const long long to = __shfl_sync(~0u, rows.v, r);
            const bool ok = (have >> r) & 1;
            if (lane % CV < vq) cp_async16((st + v_dst + i * RV * S::kValBytes) ^ (swizzle4<S::kValBytes>(i * RV) * 16), ok ? vbase + to : vbase, ok);
          }
        }
        const bool ok = rows.k >= 0;
        const int bytes = 2 * (S::GK == S::GV ? S::GK : lane < 16 ? S::GK : S::GV);
        cp_async_small(st + x_dst, ok ? xbase + rows.x : xbase, ok, bytes);
      }
      cp_async_commit();
      return have;
    };

#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) live[s] = issue(s, s, lookup(s));
    Decode4Math<S> c(a, pc);  // the queries are read while the first tokens come
    Rows rows = lookup(kStages - 1);
    int stage = 0;
    for (int step = 0; step < steps; ++step) {
      const int fill = stage == 0 ? kStages - 1 : stage - 1;  // the stage read in the last step
      __syncwarp();
      {
        const unsigned lv = issue(step + kStages - 1, fill, rows);
#pragma unroll
        for (int s = 0; s < kStages; ++s)
          if (s == fill) live[s] = lv;
      }
      rows = lookup(step + kStages);
      cp_async_wait<kStages - 1>();
      __syncwarp();
      unsigned lv = 0;
#pragma unroll
      for (int s = 0; s < kStages; ++s)
        if (s == stage) lv = live[s];
      c.step(ring + stage * S::kStageBytes, lv, pc.len - 1 - (base + step * (kDecodeWarps * kStep)), a, area);
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    cp_async_wait<0>();
    __syncthreads();  // every warp is through with its ring: it now takes the results [warp][heads][DV]
    float* res = reinterpret_cast<float*>(smem);
    c.store(res + warp * pc.heads * DV, ms[warp], ls[warp]);
    __syncthreads();
    // The four warps' results as one: into the output, the workspace, or (whole
    // items of a cluster) this CTA's part.
    float* part_s = res + kDecodeWarps * S::kHeads * DV;
    float* part = WHOLE ? nullptr : a.part + (2 * cta + (pc.starts ? 1 : 0)) * part_floats(a.item_heads, a.dv);
    const bool out = pc.starts && pc.ends;
    if (tid < pc.heads) {
      float mm = kNegInf, ll = 0.f, f[kDecodeWarps];
#pragma unroll
      for (int w = 0; w < kDecodeWarps; ++w) mm = fmaxf(mm, ms[w][tid]);
      const float mu = mm == kNegInf ? 0.f : mm;
#pragma unroll
      for (int w = 0; w < kDecodeWarps; ++w) {
        f[w] = exp2_approx(ms[w][tid] - mu);
        ll = fmaf(f[w], ls[w][tid], ll);
      }
      // Divided here, so that no sum of parts is larger than the values are; the sum goes into the maximum.
      const float inv = ll == 0.f ? 0.f : 1.f / ll;
#pragma unroll
      for (int w = 0; w < kDecodeWarps; ++w) ms[w][tid] = f[w] * inv;
      const float m_all = ll == 0.f ? kNegInf : mm + log2f(ll), l_all = ll == 0.f ? 0.f : ll == ll ? 1.f : ll;
      if constexpr (WHOLE) part_m[tid] = m_all, part_l[tid] = l_all;
      else if (!out) part[tid] = m_all, part[a.item_heads + tid] = l_all;
    }
    __syncthreads();
    T* o = static_cast<T*>(a.o) + pc.b * a.os_b + pc.h0 * a.os_h;
    for (int e = tid; e < pc.heads * DV; e += kDecodeThreads) {
      const int hd = e / DV, d = e % DV;
      if (d >= a.dv) continue;
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kDecodeWarps; ++w) sum = fmaf(ms[w][hd], res[(w * pc.heads + hd) * DV + d], sum);
      if (out) o[hd * a.os_h + d] = from_f32<T>(sum);
      else if constexpr (WHOLE) part_s[hd * DV + d] = sum;
      else part[2 * a.item_heads + hd * a.dv + d] = sum;
    }
    if constexpr (WHOLE) {
      if (a.split > 1) {  // the cluster's CTAs share the item: each joins every a.split-th value of all
        cluster_sync();
        for (int e = tid * a.split + static_cast<int>(cluster_ctarank()); e < pc.heads * DV; e += kDecodeThreads * a.split) {
          const int hd = e / DV, d = e % DV;
          if (d >= a.dv) continue;
          float m[8], mm = kNegInf, sum = 0.f, ll = 0.f;
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            m[r] = r < a.split ? ld_cluster_f32(map_shared_rank(smem_u32(part_m + hd), r)) : kNegInf;
            mm = fmaxf(mm, m[r]);
          }
          const float mu = mm == kNegInf ? 0.f : mm;
#pragma unroll
          for (int r = 0; r < 8; ++r)
            if (r < a.split) {
              const float f = exp2_approx(m[r] - mu);
              sum = fmaf(f, ld_cluster_f32(map_shared_rank(smem_u32(part_s + e), r)), sum);
              ll = fmaf(f, ld_cluster_f32(map_shared_rank(smem_u32(part_l + hd), r)), ll);
            }
          o[hd * a.os_h + d] = from_f32<T>(ll == 0.f ? 0.f : sum / ll);
        }
        cluster_sync();  // the parts are read before any CTA leaves
      }
      return;
    }
    if (!out && pc.starts && tid == 0) note_item(a, run, pc, per_seq, cta);
    at += pc.dealt;
    __syncthreads();
  }
}

template <class S>
cudaError_t launch_decode4_shape(const DecodeArgs& a, cudaStream_t s) {
  if (a.split) {
    const long long ctas = static_cast<long long>(a.B) * a.Hkv * a.chunks * a.split;
    const cudaError_t e = smem_attr_once<decode4_stream_kernel<S, true>>(S::kSmem);
    if (e != cudaSuccess) return e;
    if (ctas >= (1LL << 31)) return cudaErrorInvalidConfiguration;
    const dim3 grid(static_cast<unsigned>(ctas));
    if (a.split == 1) return launch_pdl(decode4_stream_kernel<S, true>, grid, dim3(kDecodeThreads), S::kSmem, s, a);
    return launch_pdl_cluster(decode4_stream_kernel<S, true>, grid, dim3(kDecodeThreads), S::kSmem, s, a.split, a);
  }
  const size_t smem = S::kSmem + sizeof(unsigned) * (a.B + 1);
  const cudaError_t e = smem_attr_once<decode4_stream_kernel<S, false>>(smem);
  if (e != cudaSuccess) return e;
  // After the kernel before it, not among its CTAs: this wave fills the SMs exactly (decode_stream.cuh).
  return launch_serial(decode4_stream_kernel<S, false>, dim3(a.ctas), dim3(kDecodeThreads), smem, s, a);
}

}  // namespace cb
