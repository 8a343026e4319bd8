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

// max|x| / 7 rounded to bf16, as its bits; a maximum that is not finite (top:
// the largest of the elements' bits without sign) gives NaN.  The quotient
// rounded to 24 bits lies on the same side of a tie as the exact one unless it
// is the tie: then the remainder decides.
__device__ __forceinline__ unsigned scale4_bits(unsigned top) {
  if (top >= 0x7f800000u) return kNanScale;
  const float amax = __uint_as_float(top), q = __fdiv_rn(amax, 7.f);
  const unsigned bits = __float_as_uint(q), low = bits & 0xffffu, hi = bits >> 16;
  if (low != 0x8000u) return hi + (low > 0x8000u);
  const float rest = fmaf(-7.f, q, amax);
  return hi + (rest > 0.f || (rest == 0.f && (hi & 1)));
}
__device__ __forceinline__ float bf16_value(unsigned bits) { return __uint_as_float(bits << 16); }

// x / s rounded to the nearest whole number, ties to even, for a group's scale.
// The product with 1 / s can miss a tie: the remainder x - k s, which is exact
// (both are multiples of the smaller's last bit, and it is no larger than s),
// says so.
struct Coder4 {
  float s, inv, half, up;
  __device__ __forceinline__ explicit Coder4(unsigned scale_bits) {
    s = bf16_value(scale_bits);
    up = s < 0x1p-64f ? 0x1p64f : 1.f;  // 1 / s stays finite; both products are exact
    s *= up;
    const bool some = s > 0.f;  // neither 0 nor NaN
    inv = some ? __fdividef(1.f, s) : 0.f;
    if (!some) s = 0.f, up = 0.f;
    half = some ? 0.5f * s : 1.f;
  }
  __device__ __forceinline__ unsigned nibble(float x) const {
    x = up == 0.f ? 0.f : x * up;
    float k = rintf(x * inv);
    const float r = fmaf(-k, s, x), a = fabsf(r);
    if (a > half || (a == half && (static_cast<int>(k) & 1))) k += copysignf(1.f, r);
    return static_cast<unsigned>(static_cast<int>(fminf(fmaxf(k, -7.f), 7.f)) + 8);
  }
  __device__ __forceinline__ uint32_t word(const float (&x)[8]) const {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) w |= nibble(x[i]) << (4 * i);
    return w;
  }
};

// Where token j of sequence b lies: its page, or -1 (and the error recorded).
__device__ __forceinline__ int cache_page(const PagedArgs& c, int* err, int b, long long j, int* slot) {
  const long long pg = j < 0 ? -1 : j / c.page_size;
  int page = -1;
  if (pg >= 0 && pg < c.max_pages) page = c.table[b * c.table_stride + pg];
  if (page < 0 || page >= c.num_pages) {
    atomicCAS(err, 0, 1);  // CB_ERR_INVALID_ARG
    return -1;
  }
  *slot = static_cast<int>(j - pg * c.page_size);
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
