// Values of a 4-bit cache: 32 consecutive dims of a token's head are a group
// with one scale s (bf16); an element is c s with a code c in -7..7, stored as
// the nibble c + 8.  Byte i of a row holds dim 2i in its low half and dim
// 2i + 1 in its high one.  All roundings are those of exact arithmetic, so the
// same tokens give the same bits whichever kernel stores them.
#pragma once

#include "attention_common.cuh"

namespace cb {

constexpr int kGroup4 = 32;
__host__ __device__ constexpr int scales4(int dim) { return 2 * ((dim + 2 * kGroup4 - 1) / (2 * kGroup4)); }
constexpr unsigned kNanScale = 0x7fc0u;

__device__ __forceinline__ float bf16_value(unsigned bits) { return __uint_as_float(bits << 16); }

// max|x| / 7 rounded to bf16, as its bits; a maximum that is not finite (top:
// the largest of the elements' bits without sign) gives NaN.  A quotient that is
// off by a few 2^-24 names the right bf16 numbers around it, or is so near one of
// them that either neighbour leads to it; 7 times their middle is exact, and the
// remainder's sign with it.
__device__ __forceinline__ unsigned scale4_bits(unsigned top) {
  const float amax = __uint_as_float(top);
  const unsigned lo = __float_as_uint(amax * (1.f / 7.f)) >> 16;
  const float rest = fmaf(-7.f, __uint_as_float((lo << 16) | 0x8000u), amax);
  const unsigned bits = lo + (rest > 0.f || (rest == 0.f && (lo & 1)));
  return top >= 0x7f800000u ? kNanScale : bits;
}

// x / s rounded to the nearest whole number, ties to even, for a group's scale.
// The product with 1 / s can miss a tie: the remainder x - k s, which is exact
// (both are multiples of the smaller's last bit, and it is no larger than s),
// says so.
struct Coder4 {
  float s, inv, half, up;
  unsigned bits;
  __device__ __forceinline__ explicit Coder4(unsigned scale_bits) : bits(scale_bits) {
    s = bf16_value(scale_bits);
    up = s < 0x1p-64f ? 0x1p64f : 1.f;  // 1 / s stays finite; both products are exact
    s *= up;
    const bool some = s > 0.f;  // neither 0 nor NaN
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));  // s <= max / 7: 1 / s is no subnormal
    if (!some) s = inv = 0.f;
    half = some ? 0.5f * s : __builtin_huge_valf();
  }
  __device__ __forceinline__ unsigned nibble(float x) const {
    if (s == 0.f) return 8;
    x *= up;
    float k = rintf(x * inv);
    const float r = fmaf(-k, s, x), a = fabsf(r);
    if (a > half || (a == half && (static_cast<int>(k) & 1))) k += copysignf(1.f, r);
    return static_cast<unsigned>(static_cast<int>(fminf(fmaxf(k, -7.f), 7.f)) + 8);
  }
  // Eight elements, for scales that are no subnormals: k = 7 is the most then (max / s < 7.02), and x / s + 8 comes out
  // of one FMA with 1.5 * 2^23 as that number's low bits.  Twice, with 1 / s a little too large and a little too small:
  // the two differ where x / s is a tie, or within 2^-18 of one.  bf16 elements, of 8 bits as the scale, have none of
  // those but the ties (the others are 2^-12 away), whose even side is the one that is even; fp32 ones ask nibble().
  template <bool BF16>
  __device__ __forceinline__ uint32_t word(const float (&x)[8]) const {
    constexpr float kBase = 12582920.f;  // 1.5 * 2^23 + 8
    const float more = inv * (1.f + 0x1p-19f), less = inv * (1.f - 0x1p-19f);
    bool near = up != 1.f && s != 0.f;
    uint32_t away = 0, in = 0;  // the eight nibbles, above each of them the number's other bits, which the last line takes off
#pragma unroll
    for (int i = 7; i >= 0; --i) {
      const uint32_t qa = __float_as_uint(fmaf(x[i], more, kBase)), qi = __float_as_uint(fmaf(x[i], less, kBase));
      away = away * 16u + qa, in = in * 16u + qi;
    }
    away -= 0x4b400000u * 0x11111111u, in -= 0x4b400000u * 0x11111111u;
    uint32_t w = away;
    if (BF16) {
      const uint32_t odd = (away & 0x11111111u) * 15u;
      w = (in & odd) | (away & ~odd);
    } else {
      near |= away != in;
    }
    if (near) {
      w = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) w |= nibble(x[i]) << (4 * i);
    }
    return s == 0.f ? 0x88888888u : w;
  }
};

// Where token j of sequence b lies: its page, or -1 (and the error recorded).
__device__ __forceinline__ int cache_page(const PagedArgs& c, int* err, int b, long long j, int* slot) {
  // 32 bits hold every place of a table (a division of 64 costs a hundred instructions)
  const unsigned at = j < 0 || j > 0x7fffffff ? 0x7fffffffu : static_cast<unsigned>(j);
  const unsigned pg = at / static_cast<unsigned>(c.page_size);
  int page = -1;
  if (pg < static_cast<unsigned>(c.max_pages)) page = c.table[b * c.table_stride + pg];
  if (page < 0 || page >= c.num_pages) {
    atomicCAS(err, 0, 1);  // CB_ERR_INVALID_ARG
    return -1;
  }
  *slot = static_cast<int>(at - pg * static_cast<unsigned>(c.page_size));
  return page;
}

// One element of a 4-bit row.
__device__ __forceinline__ float value4(const uint8_t* codes, const uint16_t* scales, int d) {
  const int c = (codes[d >> 1] >> (4 * (d & 1))) & 15;
  return static_cast<float>(c - 8) * bf16_value(scales[d / kGroup4]);
}
__device__ __forceinline__ const uint8_t* key_codes4(const PagedArgs& c, long long page, long long slot, int h) {
  return static_cast<const uint8_t*>(c.k) + page * c.ks_p + slot * c.ks_t + h * c.ks_h;
}
__device__ __forceinline__ const uint8_t* value_codes4(const PagedArgs& c, long long page, long long slot, int h) {
  return static_cast<const uint8_t*>(c.v) + page * c.vs_p + slot * c.vs_t + h * c.vs_h;
}
__device__ __forceinline__ const uint16_t* key_scales4(const PagedArgs& c, long long page, long long slot, int h) {
  return c.k_scale + page * c.kx_p + slot * c.kx_t + h * c.kx_h;
}
__device__ __forceinline__ const uint16_t* value_scales4(const PagedArgs& c, long long page, long long slot, int h) {
  return c.v_scale + page * c.vx_p + slot * c.vx_t + h * c.vx_h;
}

}  // namespace cb
