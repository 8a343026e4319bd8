// The streaming kernel of attention over a 4-bit cache (cb_attention_decode4),
// for rows of whole words (dims that are multiples of 8; of 32: 16-byte pieces).
// Tokens are dealt as in decode_common.cuh; a CTA's four warps walk a piece
// together, each its own 32 tokens of every 128 through its own ring of copies, as
// in decode_stream.cuh.
//
// 4.5 bits an element: at the memory's rate an SM has 97 cycles for 16 tokens of
// a key head with dims of 128, 388 issue slots and 194 of the integer pipe.  So
// codes go to the MMAs (m16n8k16, f16 operands, fp32 sums) nearly as they lie:
// the bits of a nibble, alone in 16 bits, are the f16 number code * 2^-24, and of
// the nibble above it code * 2^-20, so that two ANDs make two pairs, of whole
// bytes one; ldmatrix hands each lane whole bytes of a token (keys) or of two
// tokens' same dims (values, transposed).  What is left:
//  - the nibbles hold c + 8.  Keys: a score's share of -8 sum q comes out of one
//    MMA over the group scales (fp32: goes in as the accumulators' first values).
//    Values: one more MMA with -8 everywhere per tile, in the same step, so that
//    no sum grows with the offset.
//  - a group's scale: keys, one FMA per score and group on the group's sum;
//    values, on the weights, a set of weights per group.
//  - f16's range.  Queries are scaled by a power of two per head (2^15 above).
//    A token's largest scale goes into its weight in fp32, what its groups' are
//    beside it into f16; the running maximum is that of weight times scale, so
//    that a large value of no weight takes nothing from the others.  Products
//    below 2^-31 of the largest are lost; where that, or fp32's range, could
//    show in a group (its scales far apart from the other groups' or from its
//    first ones; so with scores and queries, below), the run is done again at its
//    end by redo_run(), in fp32 on the CUDA cores.  Asking costs 1 % (calls of 196
//    -> 198.7 us for the sequences below) to 4 % (63 -> 65.3 for 64 ragged ones);
//    with that code within the loop over pieces the former took 209.
// The MMAs add 16 products and the sum so far with all that lies 25 bits below
// the largest exponent cut off, toward zero, and a subnormal's exponent counts as
// 2^-14: a step's sums keep 15 bits below their largest term, besides the 11 of a
// weight.  For fp32 that would show, so there queries are two whole numbers of at
// most 2^11 on a common grid per head and group (hi + lo 2^-12, 24 bits below the
// group's largest element, where that is 2^-20 of the head's or more), whose
// products and sums are exact; weights are sums of two f16 numbers (22 bits),
// codes are made f16 numbers of their own size, and a step's products are added
// to O by FADDs.
//
// Measured: 16 tokens of a key head take 377 instructions, half the schedulers'
// slots are filled, and neither memory nor a pipe is: eight sequences of up to
// 131072 tokens, 8 key heads of 128, in 196 us, 0.68 of the copy rate (the bf16
// cache's 466).  The bf16 kernels of 128 dims and 8 heads are held to 128 registers
// and spill 4 to 60 bytes.  Three CTAs of three stages take as long as four of two
// (three with one stage less in flight, four with fewer registers than they want).
// fp8 MMAs, whose e4m3 subnormals the codes are as well, run as two f16 ones after
// conversions: 249 us where f16 took 205.
#pragma once

#include <cuda_fp16.h>

#include <cstring>
#include <type_traits>

#include "cache4.cuh"
#include "decode_stream.cuh"
#include "stage_ring.h"

namespace cb {

template <int BYTES>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(valid ? BYTES : 0) : "memory");
}
__device__ __forceinline__ void copy_scales(uint32_t dst, const uint16_t* src, const uint16_t* any, int count, bool valid) {
  if (count == 4) cp_async_small<8>(dst, valid ? src : any, valid);
  else cp_async_small<4>(dst, valid ? src : any, valid);
}
__device__ __forceinline__ void tma_load_4d_at(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ float4 lds_f4(uint32_t at) {
  const uint4 v = lds128(at);
  return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
}
__device__ __forceinline__ float lds_f(uint32_t at) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void sts_f(uint32_t at, float v) { asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory"); }
__device__ __forceinline__ void sts128(uint32_t at, float4 v) {
  asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<unsigned>(127 + e) << 23); }  // -126 <= e <= 127
// mbar_wait for waits of microseconds: the hardware may hold the warp for as long, so that it takes no issue slots from
// the others.
__device__ __forceinline__ bool mbar_wait_long(uint64_t* bar, uint32_t parity, const Watchdog& wd) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(20000)
      : "memory");
  return ok || mbar_wait(bar, parity, wd);
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
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
// d (16 x 8, fp32) = c + a (16 x 16, f16) * b (16 x 8, f16)
__device__ __forceinline__ void mma_f16(float (&d)[4], float c0, float c1, float c2, float c3, uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// d (16 x 8, fp32) = a (16 x 8, tf32) * b (8 x 8, tf32)
__device__ __forceinline__ void mma_tf32(float (&d)[4], float a0, float a1, float a2, float a3, float b0, float b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(__float_as_uint(a0)), "r"(__float_as_uint(a1)), "r"(__float_as_uint(a2)), "r"(__float_as_uint(a3)), "r"(__float_as_uint(b0)),
        "r"(__float_as_uint(b1)), "f"(0.f));
}
__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t half2_times(uint32_t x, float bits) {  // bits: a pair of f16 numbers
  const uint32_t y = __float_as_uint(bits);
  const __half2 h = __hmul2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&y));
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t half2_less(uint32_t x, uint32_t y) {
  const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&y));
  return *reinterpret_cast<const uint32_t*>(&h);
}
// What f16 rounding left of a pair: another pair of f16 numbers.
__device__ __forceinline__ uint32_t half2_rest(float lo, float hi, uint32_t bits) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&bits));
  return half2_bits(lo - f.x, hi - f.y);
}

constexpr uint32_t kLowNibble = 0x000f000fu, kHighNibble = 0x00f000f0u;  // times 2^-24, 2^-20
constexpr uint32_t kByte = 0x00ff00ffu, kByteMinus8 = 0x80888088u, kHighMinus8 = 0x80808080u;  // -8 (1 + 16) and -8, as they count
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
constexpr uint64_t kDrainNs = 20000000;  // a copy in flight behind a wait that ran out
constexpr int kWeightBits = 7;           // weights times scales go up to 2^15: f16's range, 2^8 above their running maximum
constexpr float kLeastScale = 0x1p-80f;  // of a token, beside its group's first: below it counts as this
constexpr float kMostScale = 0x1p100f;   // and from here on redo() has to do it
constexpr int kThin = 20;                // a group of queries that is 2^-20 of its head's largest has all its bits
constexpr float kMostScore = 0x1p20f;    // and beyond this maximum of scores
constexpr int kMostUp = 60;              // the first ones are made about 1, by 2^60 at most

template <int DK_, int DV_, int NB_, typename T_>
struct Decode4Shape {
  using T = T_;
  static constexpr int DK = DK_, DV = DV_, NB = NB_, kStep = 32, kStages = 2, kHeads = 8 * NB_;
  static constexpr int kParts = sizeof(T) == 4 ? 2 : 1;
  static constexpr int GK = DK / kGroup4, GV = DV / kGroup4;
  static constexpr int kKeyBytes = DK / 2, kValBytes = DV / 2;
  static constexpr int kStageBytes = kStep * (kKeyBytes + kValBytes), kScaleBytes = kStep * (GK + GV) * 2;
  static constexpr int kRing = kDecodeWarps * kStages * kStageBytes;
  static constexpr int kResults = 4 * (kDecodeWarps + 1) * kHeads * DV;  // the warps' and the CTA's, when a piece ends
  static constexpr int kMain = kRing > kResults ? kRing : kResults;
  // Behind the ring of codes: a step's scales as the products take them, per warp (keys' fp32, values' fp32 or f16,
  // tokens' largest, the values' multipliers); the ring of scales; queries; barriers.
  static constexpr int kArea = kStep * (2 * 16 + 4) + 32, kScales = kMain + kDecodeWarps * kArea;
  static constexpr int kQueries = kScales + kDecodeWarps * kStages * kScaleBytes, kBars = kQueries + kParts * GK * NB * 512;
  static constexpr int kSmem = kBars + kDecodeWarps * kStages * 8, kAlign = 512;  // of the copies' swizzle
  static constexpr int kCtasPerSm = decode4_ctas_per_sm(DK, DV, sizeof(T) == 2, kHeads, 0);
};

// Row r's 16-byte piece p lies at p ^ swizzle(r): ldmatrix reads one piece of eight rows.
template <int BYTES>
__device__ __forceinline__ constexpr int swizzle4(int row) {
  return BYTES == 64 ? (row >> 1) & 3 : (row >> 2) & 1;
}

template <class S, bool DIRECT>
struct Decode4Math {
  using T = typename S::T;
  static constexpr int GK = S::GK, GV = S::GV, NB = S::NB;
  // What a weight rounded below 2^-14 loses is 2^-25 at most; a group's largest product of weight and scale, when the
  // maximum is set, 2^7 times this at least.  So that is 2^-20 of it, or for fp32 2^-24.
  static constexpr float kApart = S::kParts == 1 ? 0x1p-12f : 0x1p-8f;
  int g, t4, heads;
  uint32_t k_src, v_src;  // this lane's ldmatrix rows
  // Queries as the MMAs' B operand, for each part and group: head g, dims 8 t4 + (0, 4) and (1, 5) / 16, then (2, 6) and
  // (3, 7) / 16.  In shared memory, one copy for the CTA: in registers they would cost it a neighbour.
  uint32_t queries;
  // The offsets -8 sum q. bf16: of group t4 and head 8 nb + g, as two tf32 numbers: with a key's scales as A, one MMA
  // makes a score's share of them. fp32: of every group and this thread's heads 8 nb + 2 t4 and the one after.
  float offset[NB][2], first[S::kParts == 2 ? 2 : 1][S::kParts == 2 ? GK : 1][NB][2];
  float k_mul, head_mul[NB][2];
  // The values' scales are taken times v_mul, the power of two that makes a group's first ones about 1 (0: none yet).  Those
  // lie in shared memory behind the scales' area; behind them whether the warp met what this arithmetic does not hold
  // (for the whole launch), and the largest scale that a key may have where queries are small (else infinity).  unset:
  // scales() has something to do for them.
  bool unset;
  // neg = kWeightBits - maximum of x + log2 of a token's largest scale (+infinity before the first token): weights are
  // 2^(x + neg).
  float slope[NB][2], neg[NB][2], l[NB][2], o[2 * GV][NB][4];

  // This lane's queries: dims 8 t4 .. + 8 of each group of heads 8 nb + g.  Read before the first tokens are looked up.
  struct Raw {
    T x[NB][GK][8];
  };
  static __device__ __forceinline__ void fetch(const DecodeArgs& a, const Piece& pc, Raw& raw) {
    const int g = (threadIdx.x & 31) >> 2, t4 = threadIdx.x & 3;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int hd = g + 8 * nb;
      const T* q = static_cast<const T*>(a.q) + pc.b * a.qs_b + (pc.h0 + (hd < pc.heads ? hd : 0)) * a.qs_h + 8 * t4;
#pragma unroll
      for (int i = 0; i < GK; ++i, q += 32) {
        constexpr int kPer = 16 / static_cast<int>(sizeof(T));
        uint4 w[8 / kPer] = {};
        if (hd < pc.heads && 32 * i + 8 * t4 < a.dk) {
          if (reinterpret_cast<uintptr_t>(q) % 16 == 0) {
#pragma unroll
            for (int e = 0; e < 8 / kPer; ++e) w[e] = reinterpret_cast<const uint4*>(q)[e];
          } else {
            T x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = q[e];
            memcpy(w, x, sizeof(w));
          }
        }
        memcpy(raw.x[nb][i], w, sizeof(w));
      }
    }
  }

  __device__ __forceinline__ Decode4Math(const DecodeArgs& a, const Piece& pc, const Raw& raw, uint4* q_area, uint32_t area) {
    queries = smem_u32(q_area + (threadIdx.x & 31));
    const DecodeScore score(a);
    const int lane = threadIdx.x & 31;
    g = lane >> 2, t4 = lane & 3, heads = pc.heads, unset = true;
    const int row = (lane & 7) + 8 * ((lane >> 3) & 1);
    k_src = row * S::kKeyBytes + (((lane >> 4) ^ swizzle4<S::kKeyBytes>(row)) * 16);
    v_src = row * S::kValBytes + (((lane >> 4) ^ swizzle4<S::kValBytes>(row)) * 16);
    if (lane == 0) sts128(area + 1152, make_float4(0.f, 0.f, 0.f, 0.f)), sts_f(area + 1172, __builtin_huge_valf());
    __syncwarp();
    int exponent[NB], top = -1000, thin = -1000;
    float sums[S::kParts][GK][NB];
    constexpr int kBits = S::kParts == 2 ? 11 : 15;  // queries go up to 2^kBits
    constexpr int kCodeBits = 24;                   // codes are c + 8 times 2^-kCodeBits
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      float x[GK][8], big = 0.f, of[GK];  // of: a group's largest (bf16: of this lane's dims)
#pragma unroll
      for (int i = 0; i < GK; ++i) {
        of[i] = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[i][e] = to_f32(raw.x[nb][i][e]);
          of[i] = fmaxf(of[i], fabsf(x[i][e]));
        }
        if constexpr (S::kParts == 2) {
          of[i] = fmaxf(of[i], __shfl_xor_sync(~0u, of[i], 1));
          of[i] = fmaxf(of[i], __shfl_xor_sync(~0u, of[i], 2));
        }
        big = fmaxf(big, of[i]);
      }
      if constexpr (S::kParts == 1) {
        big = fmaxf(big, __shfl_xor_sync(~0u, big, 1));
        big = fmaxf(big, __shfl_xor_sync(~0u, big, 2));
      }
      auto above = [](float m) {  // m is below 2^above; 0 for what is no number
        return m > 0.f && m < __builtin_huge_valf() ? max(static_cast<int>(__float_as_uint(m) >> 23), 1) - 126 : 0;
      };
      const int e2 = above(big);
      const float p1 = pow2((kBits - e2) / 2), p2 = pow2(kBits - e2 - (kBits - e2) / 2);
      exponent[nb] = e2 - kBits;
      if (big > 0.f) top = max(top, exponent[nb]);
#pragma unroll
      for (int i = 0; i < GK; ++i) {
        float y[8], sum[S::kParts] = {};
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = x[i][e] * p1 * p2;
        const int below = of[i] > 0.f && big < __builtin_huge_valf() ? e2 - above(of[i]) : 0;  // the head's largest
        if (below > kThin) thin = max(thin, e2);
        if constexpr (S::kParts == 1) {
          uint32_t qf[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {  // dims 8 t4 + r and r + 4; odd r: a sixteenth
            const float unit = r & 1 ? 0.0625f : 1.f;
            qf[r] = half2_bits(y[r] * unit, y[r + 4] * unit);
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&qf[r]));
            sum[0] += (f.x + f.y) / unit;
          }
          if (threadIdx.x < 32) q_area[(i * NB + nb) * 32 + lane] = make_uint4(qf[0], qf[1], qf[2], qf[3]);
        } else {
          uint32_t qf[2][4];
          const float up = pow2(min(below, kThin)), down = pow2(-min(below, kThin));
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] *= up;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float unit = r & 1 ? 0.0625f * down : down;
            const float a0 = rintf(y[r]), a1 = rintf(y[r + 4]), b0 = rintf((y[r] - a0) * 0x1p12f), b1 = rintf((y[r + 4] - a1) * 0x1p12f);
            qf[0][r] = half2_bits(a0 * unit, a1 * unit);
            qf[1][r] = half2_bits(b0 * unit, b1 * unit);
            sum[0] += (a0 + a1) * down;
            sum[1] += (b0 + b1) * down;
          }
#pragma unroll
          for (int p = 0; p < 2; ++p)
            if (threadIdx.x < 32) q_area[((p * GK + i) * NB + nb) * 32 + lane] = make_uint4(qf[p][0], qf[p][1], qf[p][2], qf[p][3]);
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
    // The heads' powers take part in their scores at the end; the keys' scales take what is above 2^60 of the largest one's,
    // so that neither leaves fp32's range where the scores do not.
    const int k_exp = max(top + kCodeBits - 60, 0);
    k_mul = pow2(k_exp);
    // A group whose queries are that far below their head's largest is off by 2^-36 of it (fp32: 2^-44) at most, which shows in
    // a score only where its keys are large: beyond this scale.
    if (__any_sync(~0u, thin != -1000)) {
      thin = __reduce_max_sync(~0u, thin);
      if (lane == 0) sts_f(area + 1172, 0x1p16f / a.scale * pow2(max(min(-thin, 126), -126)) * k_mul);
      __syncwarp();
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int from = 4 * (2 * t4 + e), hd = 8 * nb + 2 * t4 + e;
        const int he = __shfl_sync(~0u, exponent[nb], from);
        const int up = he + kCodeBits - k_exp;
        head_mul[nb][e] = up < -126 ? 0.f : pow2(up) * (score.cap ? 1.f : score.c_scale);
#pragma unroll
        for (int p = 0; p < S::kParts && S::kParts == 2; ++p)
#pragma unroll
          for (int i = 0; i < GK; ++i) first[p][i][nb][e] = __shfl_sync(~0u, sums[p][i][nb], from);
        slope[nb][e] = a.slopes && hd < heads ? a.slopes[pc.h0 + hd] * kLog2e : 0.f;
        neg[nb][e] = __builtin_huge_valf();
        l[nb][e] = 0.f;
      }
#pragma unroll
      for (int d = 0; d < 2 * GV; ++d)
#pragma unroll
        for (int r = 0; r < 4; ++r) o[d][nb][r] = 0.f;
      float f = 0.f;
#pragma unroll
      for (int i = 0; i < GK; ++i) f = t4 == i ? sums[0][i][nb] : f;
      offset[nb][0] = __uint_as_float(__float_as_uint(f) & 0xffffe000u);  // tf32's bits; the rest, of 13, as another
      offset[nb][1] = f - offset[nb][0];
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

  // Scores of 16 tokens before the heads' factors: element r is key g + 8 (r >> 1), head 8 nb + 2 t4 + (r & 1).
  __device__ __forceinline__ void scores(float (&s)[NB][4], uint32_t keys, uint32_t area) const {
    const float4 x0 = lds_f4(area + 16 * g), x1 = lds_f4(area + 16 * (g + 8));
    const float k0[4] = {x0.x, x0.y, x0.z, x0.w}, k1[4] = {x1.x, x1.y, x1.z, x1.w};
    if constexpr (S::kParts == 1) {  // a scale has bf16's 8 bits
      const float y0 = lds_f(area + 16 * g + 4 * t4), y1 = lds_f(area + 16 * (g + 8) + 4 * t4);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) mma_tf32(s[nb], y0, y1, y0, y1, offset[nb][0], offset[nb][1]);
    }
#pragma unroll
    for (int i = 0; i < GK; i += 2) {
      uint32_t w[4];  // groups i and i + 1: a word of key g and of key g + 8
      ldsm4_4((keys + k_src) ^ (i * 16), w);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t u = w[2 * j], v = w[2 * j + 1], ub = __byte_perm(u, 0, 0x4341), vb = __byte_perm(v, 0, 0x4341);
        const uint32_t uh = u & kHighNibble, vh = v & kHighNibble, ubh = ub & kHighNibble, vbh = vb & kHighNibble;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float acc[S::kParts][4];
#pragma unroll
          for (int p = 0; p < S::kParts; ++p) {
            const uint4 q = lds128(queries + ((p * GK + i + j) * NB + nb) * 512);
            float f0 = 0.f, f1 = 0.f;
            if constexpr (S::kParts == 2) f0 = first[p][i + j][nb][0], f1 = first[p][i + j][nb][1];
            mma_f16(acc[p], f0, f1, f0, f1, u & kLowNibble, v & kLowNibble, uh, vh, q.x, q.y);
            mma_f16(acc[p], half2_less(ub, ubh), half2_less(vb, vbh), ubh, vbh, q.z, q.w);
          }
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float k = r < 2 ? k0[i + j] : k1[i + j], sum = S::kParts == 2 ? fmaf(acc[S::kParts - 1][r], 0x1p-12f, acc[0][r]) : acc[0][r];
            s[nb][r] = S::kParts == 2 && i + j == 0 ? sum * k : fmaf(sum, k, s[nb][r]);
          }
        }
      }
    }
  }

  // O += weights (of 16 tokens, in s) times values; bf16: rows g of a tile take whole bytes, c + 16 c', rows g + 8 the
  // high nibble 16 c' alone, for an AND less than the low one alone; store() subtracts.  area: S::kParts == 1,
  // [token pair][group] pairs of f16 scales; else [token] four fp32 scales.
  __device__ __forceinline__ void outputs(const float (&s)[NB][4], uint32_t vals, uint32_t area) {
    constexpr bool kF16 = S::kParts == 1;
    const float4 x0 = lds_f4(area + 16 * (kF16 ? t4 : g)), x1 = lds_f4(area + 16 * (kF16 ? t4 + 4 : g + 8));
    const float c0[4] = {x0.x, x0.y, x0.z, x0.w}, c1[4] = {x1.x, x1.y, x1.z, x1.w};
    uint32_t b[NB][2];
    if constexpr (kF16)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int r = 0; r < 2; ++r) b[nb][r] = transpose8x8(half2_bits(s[nb][2 * r], s[nb][2 * r + 1]));
#pragma unroll
    for (int i = 0; i < GV; i += 2) {
      uint32_t w[4];  // groups i and i + 1: dims 4 g .. + 4 of tokens 2 t4, 2 t4 + 1 and of those + 8
      ldsm4_4t((vals + v_src) ^ (i * 16), w);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t u = w[2 * j], v = w[2 * j + 1], u8 = u >> 8, v8 = v >> 8;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float(&d0)[4] = o[2 * (i + j)][nb], (&d1)[4] = o[2 * (i + j) + 1][nb];
          if constexpr (kF16) {
            const uint32_t b0 = half2_times(b[nb][0], c0[i + j]), b1 = half2_times(b[nb][1], c1[i + j]);
            const uint32_t ub = __byte_perm(u, 0, 0x4341), vb = __byte_perm(v, 0, 0x4341);
            mma_f16(d0, u & kByte, u & kHighNibble, v & kByte, v & kHighNibble, b0, b1);
            mma_f16(d1, ub, ub & kHighNibble, vb, vb & kHighNibble, b0, b1);
            mma_f16(d0, kByteMinus8, kHighMinus8, kByteMinus8, kHighMinus8, b0, b1);
            mma_f16(d1, kByteMinus8, kHighMinus8, kByteMinus8, kHighMinus8, b0, b1);
          } else {
            const float p0 = s[nb][0] * c0[i + j], p1 = s[nb][1] * c0[i + j], p2 = s[nb][2] * c1[i + j], p3 = s[nb][3] * c1[i + j];
            uint32_t lo = half2_bits(p0, p1), hi = half2_bits(p2, p3);
            float fresh[2][4] = {};
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              if (p) lo = half2_rest(p0, p1, lo), hi = half2_rest(p2, p3, hi);
              const uint32_t b0 = transpose8x8(lo), b1 = transpose8x8(hi);
              mma_f16(fresh[0], low_codes(u), high_codes(u), low_codes(v), high_codes(v), b0, b1);
              mma_f16(fresh[1], low_codes(u8), high_codes(u8), low_codes(v8), high_codes(v8), b0, b1);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) d0[r] += fresh[0][r], d1[r] += fresh[1][r];
          }
        }
      }
    }
  }

  // A token's scales of a step: this lane's, 0 behind the last group's.
  template <bool FULL>
  static __device__ __forceinline__ float4 load_scales(uint32_t at, int groups, int dim, unsigned lv) {
    uint32_t w0, w1 = 0;
    if (groups == 4) asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w0), "=r"(w1) : "r"(at) : "memory");
    else asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w0) : "r"(at) : "memory");
    if (!FULL && !((lv >> (threadIdx.x & 31)) & 1)) w0 = w1 = 0;
    if (dim <= 32) w0 &= 0xffffu;
    if (dim <= 96) w1 = dim <= 64 ? 0 : w1 & 0xffffu;
    return make_float4(__uint_as_float(w0 << 16), __uint_as_float(w0 & 0xffff0000u), __uint_as_float(w1 << 16),
                       __uint_as_float(w1 & 0xffff0000u));
  }

  // Whether this lane's token has scales that f16 weights and the sums do not hold (s: the groups', times their
  // multipliers; most: the largest as it goes into the weights): one that left fp32's range beside the first ones, or
  // groups' that are far apart.  The maximum is that of weight times a token's largest scale, for all groups, so that where
  // such a token sets it another group's products would be rounded, or lost, below f16's range.  Asked where a maximum
  // grows or a group's multiplier is set: between those what a group loses is small beside what it had then.
  // Its run (whole items: it) is then done again, by redo_run() or redo().
  __device__ __forceinline__ void ask(const float (&s)[4], const float (&mul)[4], float most, uint32_t area) const {
    float least = __builtin_huge_valf(), top = 0.f;
#pragma unroll
    for (int i = 0; i < GV; ++i)
      if (mul[i] != 0.f) least = fminf(least, s[i]), top = fmaxf(top, s[i]);  // else nothing but zeros so far
    if (!(most < kMostScale) || (top > 0.f && least < most * kApart)) set_beyond(area);
  }
  static __device__ __forceinline__ void set_beyond(uint32_t area) { sts_f(area + 1168, 1.f); }

  // The step's scales as the products take them, a token per lane: area [32] keys', then values'.
  template <bool FULL>
  __device__ __forceinline__ void scales(uint32_t raw, unsigned lv, const DecodeArgs& a, uint32_t area) {
    const int lane = threadIdx.x & 31;
    float4 k = load_scales<FULL>(raw + lane * GK * 2, GK, a.dk, lv), v = load_scales<FULL>(raw + S::kStep * GK * 2 + lane * GV * 2, GV, a.dv, lv);
    k.x *= k_mul, k.y *= k_mul, k.z *= k_mul, k.w *= k_mul;
    sts128(area + 16 * lane, k);
    float vs[4] = {v.x, v.y, v.z, v.w};
    float4 mul = lds_f4(area + 1152);
    float v_mul[4] = {mul.x, mul.y, mul.z, mul.w};
    bool fresh = false;
    if (unset) {
      const float most_key = lds_f(area + 1172);  // of a group of queries far below their head's largest
      unset = most_key < __builtin_huge_valf();
      if (fmaxf(fmaxf(k.x, k.y), fmaxf(k.z, k.w)) > most_key) set_beyond(area);
#pragma unroll
      for (int i = 0; i < GV; ++i) {
        if (v_mul[i] != 0.f || i * kGroup4 >= a.dv) continue;
        const unsigned top = __reduce_max_sync(~0u, vs[i] < __builtin_huge_valf() ? __float_as_uint(vs[i]) : 0);
        if (top) v_mul[i] = pow2(min(126 - static_cast<int>(top >> 23), kMostUp)), fresh = true;  // below 1 then
        else unset = true;
      }
      __syncwarp();
      if (lane == 0) sts128(area + 1152, make_float4(v_mul[0], v_mul[1], v_mul[2], v_mul[3]));
    }
    float most = kLeastScale;
#pragma unroll
    for (int i = 0; i < GV; ++i) {
      vs[i] *= v_mul[i];
      most = fmaxf(most, vs[i]);  // not NaN
    }
    if (fresh) ask(vs, v_mul, most, area);
    sts_f(area + 1024 + 4 * lane, most);
    v = make_float4(vs[0], vs[1], vs[2], vs[3]);
    if constexpr (S::kParts == 2) {
      sts128(area + 512 + 16 * lane, v);
    } else {
      // Beside the token's largest, which goes into the weights.  Tokens' pairs side by side: an even lane takes groups 0
      // and 1 of the pair, an odd one 2 and 3.
      float less;
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(less) : "f"(most));
      v.x *= less, v.y *= less, v.z *= less, v.w *= less;
      const uint32_t h01 = half2_bits(v.x, v.y), h23 = half2_bits(v.z, v.w);
      const bool odd = lane & 1;
      const uint32_t own = odd ? h23 : h01, other = __shfl_xor_sync(~0u, odd ? h01 : h23, 1);
      const uint32_t lo = odd ? other : own, hi = odd ? own : other;
      asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(area + 512 + 8 * lane), "r"(__byte_perm(lo, hi, 0x5410)),
                   "r"(__byte_perm(lo, hi, 0x7632))
                   : "memory");
    }
    __syncwarp();
  }

  // 32 tokens of a stage, codes at st, scales at raw; bit x of lv: token x exists (FULL: all do); far: the first one's
  // distance from the query.
  // DIRECT: no cap and no bias.
  template <bool FULL>
  __device__ __forceinline__ void step(uint32_t st, uint32_t raw, unsigned lv, int far, const DecodeArgs& a, uint32_t area) {
    scales<FULL>(raw, lv, a, area);
    float s[2][NB][4];
    const bool second = FULL || (lv >> 16) != 0;  // there are tokens in the second half
    scores(s[0], st, area);
    if (second) {
      scores(s[1], st + 16 * S::kKeyBytes, area + 256);
    } else {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int r = 0; r < 4; ++r) s[1][nb][r] = 0.f;
    }
    // What the exponential takes: x + neg, x = log2(e) * score.
    float y[2][NB][4], lsum[NB][2];
    if constexpr (!DIRECT) {
      const DecodeScore score(a);
      const float dist = static_cast<float>(far - g);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int r = 0; r < 4; ++r) s[h][nb][r] *= head_mul[nb][r & 1];
        if (score.cap) score(s[h]);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int r = 0; r < 4; ++r) s[h][nb][r] = fmaf(-slope[nb][r & 1], dist - 16.f * h - 8.f * (r >> 1), s[h][nb][r]);
      }
    }
    auto exponents = [&](const float (&add)[NB][2]) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            y[h][nb][r] = DIRECT ? fmaf(s[h][nb][r], head_mul[nb][r & 1], add[nb][r & 1]) : s[h][nb][r] + add[nb][r & 1];
            if (!FULL && !((lv >> (g + 8 * (r >> 1) + 16 * h)) & 1)) y[h][nb][r] = kNegInf;
          }
    };
    float most[2][2];  // the tokens' largest scales
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 2; ++e) most[h][e] = lds_f(area + 1024 + 4 * (16 * h + 8 * e + g));
    bool grow = false;
    auto weights = [&](const float (&add)[NB][2]) {  // y: weights times the largest scales; lsum: of the weights
      exponents(add);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        lsum[nb][0] = lsum[nb][1] = 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float p = exp2_approx(y[h][nb][r]), w = p * most[h][r >> 1];
            lsum[nb][r & 1] += p;
            grow |= !(w <= 0x1p15f);
            y[h][nb][r] = S::kParts == 1 ? w : p;
          }
      }
    };
    weights(neg);
    if (__any_sync(~0u, grow)) {
      {  // An infinite scale makes every weight grow (or NaN): it is met here.
        const int lane = threadIdx.x & 31;
        const float4 v = load_scales<FULL>(raw + S::kStep * GK * 2 + lane * GV * 2, GV, a.dv, lv), mul = lds_f4(area + 1152);
        ask({v.x * mul.x, v.y * mul.y, v.z * mul.z, v.w * mul.w}, {mul.x, mul.y, mul.z, mul.w}, lds_f(area + 1024 + 4 * lane), area);
      }
      float zero[NB][2], f[NB][2], now[NB][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) zero[nb][0] = zero[nb][1] = 0.f;
      exponents(zero);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = kNegInf;
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i) x = fmaxf(x, y[h][nb][2 * i + e] + __log2f(most[h][i]));
          x = fmaxf(x, __shfl_xor_sync(~0u, x, 4));
          x = fmaxf(x, __shfl_xor_sync(~0u, x, 8));
          x = fmaxf(x, __shfl_xor_sync(~0u, x, 16));
          // Before the first token the maximum is -infinity: what is multiplied then is 0.
          const float was = kWeightBits - neg[nb][e], mn = fmaxf(was, x);
          // Without a cap the exponent takes a score before its rounding, the maximum after it: more apart than f16 has room
          // for, where scores are large.
          if (DIRECT && mn > kNegInf && !(fabsf(mn) <= kMostScore)) set_beyond(area);
          const float root = was == kNegInf ? 1.f : exp2_approx(0.5f * (was - mn));
          f[nb][e] = root * root;
          neg[nb][e] = kWeightBits - mn;
          now[nb][e] = mn == kNegInf ? 0.f : neg[nb][e];
          l[nb][e] = l[nb][e] * root * root;  // in two steps: with scales far above the first ones the square may be 0
        }
      rescale(f);
      weights(now);
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) l[nb][0] += lsum[nb][0], l[nb][1] += lsum[nb][1];
    const uint32_t vals = st + S::kStep * S::kKeyBytes;
    outputs(y[0], vals, area + 512);
    if (second) outputs(y[1], vals + 16 * S::kValBytes, area + 512 + (S::kParts == 1 ? 128 : 256));
  }

  // This warp's results: res[heads][DV] divided by their sum of weights (so they are no larger than the values are),
  // the maxima with that sum in them, and sums of 1 (0: no token).
  __device__ __forceinline__ void store(float* res, float* ms, float* ls, uint32_t area) {
    const float4 mul = lds_f4(area + 1152);
    const float v_mul[4] = {mul.x, mul.y, mul.z, mul.w};
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float y = l[nb][e];
        y += __shfl_xor_sync(~0u, y, 4);
        y += __shfl_xor_sync(~0u, y, 8);
        y += __shfl_xor_sync(~0u, y, 16);
        const int hd = 8 * nb + 2 * t4 + e;
        if (g == 0) ms[hd] = y == 0.f ? kNegInf : log2f(y) - neg[nb][e], ls[hd] = y == 0.f ? 0.f : y == y ? 1.f : y;
        const float inv = y == 0.f ? 0.f : 1.f / y;
        if (hd < heads)
#pragma unroll
          for (int i = 0; i < GV; ++i) {
            const int up = v_mul[i] == 0.f ? 0 : 127 - static_cast<int>(__float_as_uint(v_mul[i]) >> 23);
            // in two steps, as the power may be no number
            const float lo1 = pow2(up / 2) * inv, lo2 = pow2(up - up / 2 + (S::kParts == 1 ? 24 : 0)), hi2 = S::kParts == 1 ? lo2 * 0.0625f : lo2;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float hi = o[2 * i + j][nb][2 + e], lo = S::kParts == 1 ? o[2 * i + j][nb][e] - hi : o[2 * i + j][nb][e];
              *reinterpret_cast<float2*>(res + hd * S::DV + 32 * i + 4 * g + 2 * j) = make_float2(lo * lo1 * lo2, hi * lo1 * hi2);
            }
          }
      }
  }
};

// The tokens of one warp of a piece: 32 (the first `take` of them) of every 128 from `base` on.
struct Share {
  int b, hk, h0, heads, len, steps, take;
  unsigned base, first, limit;
  __device__ __forceinline__ Share(const Piece& pc, int warp, int take_)
      : b(pc.b), hk(pc.hk), h0(pc.h0), heads(pc.heads), len(pc.len), steps((pc.tiles * kDecodeTile + kDecodeWarps * 32 - 1) / (kDecodeWarps * 32)),
        take(take_), base(static_cast<unsigned>(pc.tile0) * kDecodeTile + warp * take_), first(pc.lo),
        limit(min(static_cast<unsigned>(pc.hi), static_cast<unsigned>(pc.tile0 + pc.tiles) * kDecodeTile)) {}
};

// A share from the definition, in fp32 on the CUDA cores, for what the products of f16 weights cannot hold: a token per
// lane for the scores, four dims per lane for the values, two heads at a time.  Results as Decode4Math::store() leaves
// them.  Weights are taken times 2^-32, so that sums of the largest values stay finite.  Where every run is done again the
// file head's ragged and long sequences take 9 and 14 times as long (582 and 2833 us; four heads at a time 432 and 2044,
// but the long ones' main loop, which the compiler then treats otherwise, 204, not 198.7).
template <typename T>
__device__ __noinline__ void redo(const DecodeArgs& a, const Share w, float* res, int ld, float* ms, float* ls) {
  constexpr int kAtOnce = 2, kAhead = 8;  // heads; tokens whose values are in flight
  constexpr float kLess = 32.f;
  const int lane = threadIdx.x & 31, dim = 4 * lane;
  const DecodeScore score(a);
  for (int h = 0; h < w.heads; h += kAtOnce) {
    const int heads = min(kAtOnce, w.heads - h);  // the others repeat the last one
    const T* q[kAtOnce];
    float slope[kAtOnce], m[kAtOnce], mu[kAtOnce], l[kAtOnce], o[kAtOnce][4];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int hd = w.h0 + h + min(i, heads - 1);
      q[i] = static_cast<const T*>(a.q) + w.b * a.qs_b + hd * a.qs_h;
      slope[i] = a.slopes ? a.slopes[hd] * kLog2e : 0.f;
      m[i] = kNegInf, mu[i] = l[i] = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    }
    for (int step = 0; step < w.steps; ++step) {
      const unsigned j = w.base + step * (kDecodeWarps * 32) + lane;
      int page = -1, slot = 0;
      if (lane < w.take && j >= w.first && j < w.limit) page = token_page(a, w.b, static_cast<int>(j), &slot);
      float x[kAtOnce][1] = {}, p[kAtOnce];
      if (page >= 0) {
        const uint8_t* codes = key_codes4(a.cache, page, slot, w.hk);
        const uint16_t* scales = key_scales4(a.cache, page, slot, w.hk);
#pragma unroll 2
        for (int d = 0; d < a.dk; d += 8) {
          const uint32_t c = *reinterpret_cast<const uint32_t*>(codes + d / 2);
          const float s = bf16_value(scales[d / kGroup4]);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float k = (static_cast<int>((c >> (4 * e)) & 15u) - 8) * s;
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) x[i][0] = fmaf(to_f32(q[i][d + e]), k, x[i][0]);
          }
        }
      }
      score(x);
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const float y = page < 0 ? kNegInf : fmaf(-slope[i], static_cast<float>(w.len - 1 - static_cast<int>(j)), x[i][0]);
        float top = y;
        for (int n = 16; n; n >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, n));
        const float was = m[i];
        m[i] = fmaxf(m[i], top), mu[i] = m[i] == kNegInf ? 0.f : m[i];
        const float f = exp2_approx(was - mu[i]);
        p[i] = page < 0 ? 0.f : exp2_approx(y - mu[i] - kLess);
        float sum = p[i];
        for (int n = 16; n; n >>= 1) sum += __shfl_xor_sync(~0u, sum, n);
        l[i] = fmaf(l[i], f, sum);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] *= f;
      }
      if (!__any_sync(~0u, page >= 0)) continue;
      for (int t0 = 0; t0 < 32; t0 += kAhead) {
        unsigned c[kAhead], s[kAhead];
#pragma unroll
        for (int t = 0; t < kAhead; ++t) {
          const int pg = __shfl_sync(~0u, page, t0 + t), sl = __shfl_sync(~0u, slot, t0 + t);
          c[t] = s[t] = 0;  // a token that does not exist: its weight is 0 too
          if (pg >= 0 && dim < a.dv) {
            c[t] = *reinterpret_cast<const uint16_t*>(value_codes4(a.cache, pg, sl, w.hk) + dim / 2);
            s[t] = value_scales4(a.cache, pg, sl, w.hk)[dim / kGroup4];
          }
        }
#pragma unroll
        for (int t = 0; t < kAhead; ++t) {
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = (static_cast<int>((c[t] >> (4 * e)) & 15u) - 8) * bf16_value(s[t]);
#pragma unroll
          for (int i = 0; i < kAtOnce; ++i) {
            const float pt = __shfl_sync(~0u, p[i], t0 + t);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] = fmaf(pt, v[e], o[i][e]);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      if (i >= heads) break;
      const int hd = h + i;
      if (lane == 0) ms[hd] = l[i] == 0.f ? kNegInf : mu[i] + kLess + log2f(l[i]), ls[hd] = l[i] == 0.f ? 0.f : l[i] == l[i] ? 1.f : l[i];
      const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
      if (dim < a.dv) *reinterpret_cast<float4*>(res + hd * ld + dim) = make_float4(o[i][0] * inv, o[i][1] * inv, o[i][2] * inv, o[i][3] * inv);
    }
  }
}

// All pieces of a CTA's run again, by all its threads; where a warp has met what it does not hold.
template <typename T>
__device__ __noinline__ void redo_run(const DecodeArgs& a, const unsigned* prefix, float* res, int ld, float* ms, float* ls, int width) {
  const int tid = threadIdx.x, warp = tid >> 5, per_seq = a.Hkv * a.chunks;
  const long long total = static_cast<long long>(prefix[a.B]) * per_seq, cta = blockIdx.x;
  const Run run{total, min(static_cast<long long>(gridDim.x), total)};
  long long at = run.begin(cta);
  const long long end = run.begin(cta + 1);
  int b = find_seq(a, prefix, per_seq, at);
  while (at < end) {
    const Piece pc = next_piece(a, prefix, per_seq, at, end, &b);
    redo<T>(a, Share{pc, warp, 32}, res + warp * pc.heads * ld, ld, ms + warp * width, ls + warp * width);
    __syncthreads();
    const bool out = pc.starts && pc.ends;
    float* part = a.part + (2 * cta + (pc.starts ? 1 : 0)) * part_floats(a.item_heads, a.dv);
    T* o = static_cast<T*>(a.o) + pc.b * a.os_b + pc.h0 * a.os_h;
    for (int e = tid; e < pc.heads * a.dv; e += kDecodeThreads) {
      const int hd = e / a.dv, d = e % a.dv;
      float m = kNegInf, l = 0.f, sum = 0.f;
      for (int w = 0; w < kDecodeWarps; ++w) m = fmaxf(m, ms[w * width + hd]);
      const float mu = m == kNegInf ? 0.f : m;
      for (int w = 0; w < kDecodeWarps; ++w) l = fmaf(exp2_approx(ms[w * width + hd] - mu), ls[w * width + hd], l);
      const float inv = l == 0.f ? 0.f : 1.f / l;
      for (int w = 0; w < kDecodeWarps; ++w) sum = fmaf(exp2_approx(ms[w * width + hd] - mu) * inv, res[(w * pc.heads + hd) * ld + d], sum);
      if (out) o[hd * a.os_h + d] = from_f32<T>(sum);
      else part[2 * a.item_heads + hd * a.dv + d] = sum;
      if (!out && d == 0) part[hd] = l == 0.f ? kNegInf : m + log2f(l), part[a.item_heads + hd] = l == 0.f ? 0.f : l == l ? 1.f : l;
    }
    __syncthreads();
    at += pc.dealt;
  }
}
__device__ __forceinline__ bool beyond4(uint32_t area) { return lds_f(area + 1168) != 0.f; }

// TMA: pages of a multiple of 16 slots, whose codes come in boxes of 16 rows (maps: bytes of a row, slots, heads,
// pages; swizzled as swizzle4 says); else each lane copies 16-byte pieces, or words.  Scales, a token per lane, come
// by cp.async in any case.
template <class S, bool WHOLE, bool TMA, bool DIRECT>
__global__ void __launch_bounds__(kDecodeThreads, S::kCtasPerSm)
    decode4_stream_kernel(const __grid_constant__ DecodeArgs a, const Units4 units, const __grid_constant__ Maps4 maps) {
  using T = typename S::T;
  constexpr int DV = S::DV, kStep = S::kStep, kStages = S::kStages;
  static_assert(S::DK == S::DV, "keys and values lie alike in a stage");
  constexpr int CK = S::kKeyBytes / 16, RK = 32 / CK;  // 16-byte pieces of a row; rows of a warp-wide copy
  extern __shared__ __align__(128) uint8_t smem_raw[];
  __shared__ float ms[kDecodeWarps][S::kHeads], ls[kDecodeWarps][S::kHeads];
  __shared__ float part_m[S::kHeads], part_l[S::kHeads];
  __shared__ int abort_flag;
  uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & (S::kAlign - 1));

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int kq = a.dk / kGroup4, vq = a.dv / kGroup4;  // 16-byte pieces per row; what the ring's others hold meets queries of 0
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kBars) + warp * kStages;
  if constexpr (TMA) {
    if (tid == 0) abort_flag = 0;
    if (lane == 0) {
      for (int s = 0; s < kStages; ++s) mbar_init(bars + s, 2);  // the lanes that copy
      fence_mbar_init();
    }
    __syncthreads();
  }
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
  const uint32_t raw_ring = smem_u32(smem + S::kScales + warp * kStages * S::kScaleBytes);
  const uint32_t area = smem_u32(smem + S::kMain + warp * S::kArea);
  const uint32_t k_dst = (lane / CK) * S::kKeyBytes + (((lane % CK) ^ swizzle4<S::kKeyBytes>(lane / CK)) * 16);
  const int kg = scales4(a.dk), vg = scales4(a.dv);  // scales of a row, 2 or 4; a row of the ring has room for GK, GV
  const bool same = units.k_p == units.v_p && units.k_t == units.v_t;  // one offset serves both
  const bool same_x = units.kx_p == units.vx_p && units.kx_t == units.vx_t;
  // from a lane's token to its next one, without a division per step
  const int adv_pg = kDecodeWarps * kStep / a.cache.page_size, adv_slot = kDecodeWarps * kStep - adv_pg * a.cache.page_size;
  const Watchdog wd{a.err, &abort_flag, a.timeout_ns};
  StageRing<kStages> flight;
  bool alive = true;    // no wait has run out: else the warp copies and computes nothing more

  if (lane == 0) sts_f(area + 1168, 0.f);

  while (at < end) {
    Piece pc;
    if constexpr (WHOLE) pc = whole_piece(a, per_seq);
    else pc = next_piece(a, prefix, per_seq, at, end, &b);
    const char* kbase = static_cast<const char*>(a.cache.k) + pc.hk * a.cache.ks_h + (lane % CK) * 16;
    const char* vbase = static_cast<const char*>(a.cache.v) + pc.hk * a.cache.vs_h + (lane % CK) * 16;
    const unsigned kx_head = pc.hk * units.kx_h, vx_head = pc.hk * units.vx_h;

    // A single tile goes to all four warps, 16 tokens each, where it is all that the CTA has: half the chain.
    const int take = WHOLE && pc.tiles == 1 ? kDecodeTile / kDecodeWarps : kStep;
    const unsigned base = static_cast<unsigned>(pc.tile0) * kDecodeTile + warp * take;  // may pass 2^31
    const int steps = (pc.tiles * kDecodeTile + kDecodeWarps * kStep - 1) / (kDecodeWarps * kStep);
    const unsigned first = pc.lo;
    const unsigned limit = min(static_cast<unsigned>(pc.hi), static_cast<unsigned>(pc.tile0 + pc.tiles) * kDecodeTile);
    // Lanes look the step's tokens up, one step before their copies are issued: page (-1: none that the piece needs;
    // TMA: none that the 16 tokens around need) and slot.
    struct Place {
      int page, slot;
    };
    const int* table = a.cache.table + pc.b * a.cache.table_stride;
    unsigned j = base + lane;
    int pg = static_cast<int>(j / static_cast<unsigned>(a.cache.page_size)), slot = static_cast<int>(j - static_cast<unsigned>(pg) * a.cache.page_size);
    auto lookup = [&](int step) {  // once for each step, in order
      Place r{-1, slot};
      const bool need = TMA ? (j | 15) >= first && (j & ~15u) < limit : j >= first && j < limit && (!WHOLE || lane < take);
      if (step < steps && need) {
        r.page = table[pg];
        if (static_cast<unsigned>(r.page) >= static_cast<unsigned>(a.cache.num_pages)) {
          atomicCAS(a.err, 0, 1);  // CB_ERR_INVALID_ARG
          r.page = -1;
        }
      }
      j += kDecodeWarps * kStep;
      pg += adv_pg, slot += adv_slot;
      if (slot >= a.cache.page_size) slot -= a.cache.page_size, ++pg;
      return r;
    };
    auto issue = [&](int step, int stage, const Place& at_) {
      const unsigned token = base + step * (kDecodeWarps * kStep) + lane;
      const bool ok = at_.page >= 0 && (!TMA || (token >= first && token < limit));
      const unsigned have = __ballot_sync(~0u, ok);
      if (step < steps && alive) {
        const uint32_t st = ring + stage * S::kStageBytes, raw = raw_ring + stage * S::kScaleBytes;
        if constexpr (TMA) {
          if ((lane & 15) == 0) {
            uint64_t* bar = bars + stage;
            if (at_.page >= 0) {
              mbar_arrive_expect_tx(bar, 16 * (S::kKeyBytes + S::kValBytes));
              tma_load_4d_at(st + lane * S::kKeyBytes, &maps.k, bar, 0, at_.slot, pc.hk, at_.page);
              tma_load_4d_at(st + kStep * S::kKeyBytes + lane * S::kValBytes, &maps.v, bar, 0, at_.slot, pc.hk, at_.page);
            } else {
              mbar_arrive(bar);
            }
          }
        } else {
          const unsigned k_off = at_.page * units.k_p + at_.slot * units.k_t;
          const unsigned v_off = same ? k_off : at_.page * units.v_p + at_.slot * units.v_t;
          auto copies = [&](auto full) {
            constexpr bool kFull = decltype(full)::value;
#pragma unroll
            for (int i = 0; i < kStep / RK; ++i) {
              const int r = i * RK + lane / CK;
              const unsigned long long off = 16ull * __shfl_sync(~0u, k_off, r), to = same ? off : 16ull * __shfl_sync(~0u, v_off, r);
              const bool some = kFull || ((have >> r) & 1);
              const uint32_t dst = (st + k_dst + i * RK * S::kKeyBytes) ^ (swizzle4<S::kKeyBytes>(i * RK) * 16);
              if (lane % CK < kq) cp_async16(dst, some ? kbase + off : kbase, some);
              if (lane % CK < vq) cp_async16(dst + kStep * S::kKeyBytes, some ? vbase + to : vbase, some);
            }
          };
          if (units.bytes == 4) {  // words, where rows are no 16-byte pieces
            constexpr int WK = S::kKeyBytes / 4;
            const int w = lane % WK;
            const char* kw = kbase - (lane % CK) * 16;
            const char* vw = vbase - (lane % CK) * 16;
#pragma unroll 4
            for (int i = 0; i < WK; ++i) {
              const int r = (i * 32 + lane) / WK;
              const unsigned long long off = 4ull * __shfl_sync(~0u, k_off, r) + 4 * w, to = 4ull * __shfl_sync(~0u, v_off, r) + 4 * w;
              const bool some = (have >> r) & 1;
              const uint32_t dst = st + r * S::kKeyBytes + (((w >> 2) ^ swizzle4<S::kKeyBytes>(r)) * 16) + (w & 3) * 4;
              if (w < a.dk / 8) cp_async_small<4>(dst, some ? kw + off : kw, some);
              if (w < a.dv / 8) cp_async_small<4>(dst + kStep * S::kKeyBytes, some ? vw + to : vw, some);
            }
          } else if (have == ~0u) {
            copies(std::true_type{});
          } else {
            copies(std::false_type{});
          }
        }
        const unsigned kx = at_.page * units.kx_p + at_.slot * units.kx_t;
        const unsigned vx = same_x ? kx : at_.page * units.vx_p + at_.slot * units.vx_t;
        const unsigned long long k_at = static_cast<unsigned long long>(kx + kx_head) * kg, v_at = static_cast<unsigned long long>(vx + vx_head) * vg;
        copy_scales(raw + lane * S::GK * 2, a.cache.k_scale + k_at, a.cache.k_scale, kg, ok);
        copy_scales(raw + kStep * S::GK * 2 + lane * S::GV * 2, a.cache.v_scale + v_at, a.cache.v_scale, vg, ok);
      }
      cp_async_commit();
      return have;
    };

    typename Decode4Math<S, DIRECT>::Raw queries;
    Decode4Math<S, DIRECT>::fetch(a, pc, queries);
    unsigned live[kStages - 1];  // of the next steps: bit x, token x exists
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) live[s] = issue(s, s, lookup(s));
    Decode4Math<S, DIRECT> c(a, pc, queries, reinterpret_cast<uint4*>(smem + S::kQueries), area);
    __syncthreads();
    Place place = lookup(kStages - 1);
    int stage = 0;
    for (int step = 0; step < steps; ++step) {
      const int fill = stage == 0 ? kStages - 1 : stage - 1;  // the stage read in the last step
      __syncwarp();
      const unsigned lv = live[0], next = issue(step + kStages - 1, fill, place);
#pragma unroll
      for (int s = 0; s + 1 < kStages - 1; ++s) live[s] = live[s + 1];
      live[kStages - 2] = next;
      place = lookup(step + kStages);
      cp_async_wait<kStages - 1>();
      if constexpr (TMA) {
        const bool issued = alive;  // once a wait has run out, nothing is any more
        if (alive) alive = mbar_wait_long(bars + stage, flight.parity(stage), wd);
        alive = __all_sync(~0u, alive);
        if (alive) flight.waited(stage);
        else if (issued) flight.in_flight(stage, step, steps, [&](int s, unsigned parity) { mbar_wait_drain(bars + s, parity, kDrainNs); });
      }
      __syncwarp();
      const int far = static_cast<int>(pc.len - 1 - (base + step * (kDecodeWarps * kStep)));
      const uint32_t st = ring + stage * S::kStageBytes, raw = raw_ring + stage * S::kScaleBytes;
      if (TMA && !alive) break;
      if (lv == ~0u) c.template step<true>(st, raw, lv, far, a, area);
      else if (lv) c.template step<false>(st, raw, lv, far, a, area);
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    cp_async_wait<0>();
    __syncthreads();  // every warp is through with its ring: it now takes the results [warp][heads][DV]
    float* res = reinterpret_cast<float*>(smem);
    if (WHOLE && beyond4(area))
      redo<T>(a, Share{pc, warp, take}, res + warp * pc.heads * DV, DV, ms[warp], ls[warp]);
    else
      c.store(res + warp * pc.heads * DV, ms[warp], ls[warp], area);
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
    if constexpr (TMA) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the results' bytes take copies again
    __syncthreads();
  }
  if constexpr (!WHOLE) {
    bool again = false;
    for (int w = 0; w < kDecodeWarps; ++w) again |= beyond4(area + (w - warp) * S::kArea);
    if (again) redo_run<T>(a, prefix, reinterpret_cast<float*>(smem), DV, ms[0], ls[0], S::kHeads);
  }
}

template <class S, bool WHOLE, bool TMA>
cudaError_t launch_decode4_kernel(const DecodeArgs& a, const Units4& u, const Maps4& maps, cudaStream_t s) {
  const bool direct = a.softcap == 0.f && !a.slopes;
  auto* kernel = direct ? decode4_stream_kernel<S, WHOLE, TMA, true> : decode4_stream_kernel<S, WHOLE, TMA, false>;
  const size_t smem = S::kSmem + S::kAlign + (WHOLE ? 0 : sizeof(unsigned) * (a.B + 1));
  const cudaError_t e = direct ? smem_attr_once<decode4_stream_kernel<S, WHOLE, TMA, true>>(smem)
                               : smem_attr_once<decode4_stream_kernel<S, WHOLE, TMA, false>>(smem);
  if (e != cudaSuccess) return e;
  // Runs go after the kernel before them, not among its CTAs: this wave fills the SMs exactly (decode_stream.cuh).
  if (!WHOLE) return launch_serial(kernel, dim3(a.ctas), dim3(kDecodeThreads), smem, s, a, u, maps);
  const long long ctas = static_cast<long long>(a.B) * a.Hkv * a.chunks * a.split;
  if (ctas >= (1LL << 31)) return cudaErrorInvalidConfiguration;
  const dim3 grid(static_cast<unsigned>(ctas));
  if (a.split == 1) return launch_pdl(kernel, grid, dim3(kDecodeThreads), smem, s, a, u, maps);
  return launch_pdl_cluster(kernel, grid, dim3(kDecodeThreads), smem, s, a.split, a, u, maps);
}

// maps: runs over pages whose codes TMA can copy; else null.
template <class S>
cudaError_t launch_decode4_shape(const DecodeArgs& a, const Units4& u, const Maps4* maps, cudaStream_t s) {
  if (a.split) return launch_decode4_kernel<S, true, false>(a, u, Maps4{}, s);
  return maps ? launch_decode4_kernel<S, false, true>(a, u, *maps, s) : launch_decode4_kernel<S, false, false>(a, u, Maps4{}, s);
}

}  // namespace cb
