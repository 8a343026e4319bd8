// Norms of query and key heads and rotary positions of several axes in one pass
// (cb_norm_rotate).
//
// Per token and head:  y = x * rsqrt(mean x^2 + eps) * w, then pairs of dims
// turn by pos[axis] * freq.  Every element is read once and written once; the
// angles of a token serve all its heads.
//
// Angles: a frequency is kept as a fraction of a turn in 64-bit fixed point,
// u = freq / (2 pi) * 2^64, and pos * u, wrapped as integers wrap, is the angle
// in turns with every whole turn gone: exact to |pos| (freq / 2 + 1) 2^-64
// turns, 2^-32 at the farthest position, where an fp32 product of a position of
// 10^5 is off by 2^-8 radians.  What is left, in [-1/2, 1/2) turn, goes to sincospif.
#include <cuda_bf16.h>

#include "attention_common.cuh"
#include "launch_util.h"
#include "ptx.cuh"

namespace cb {

namespace {

constexpr int kWarps = 4;
constexpr int kMaxPairs = 64;

// freq / (2 pi) as a 64-bit fraction of a turn; freq is finite.
__device__ __forceinline__ unsigned long long turn_of(float freq) {
  constexpr unsigned long long kInv2Pi = 0x28BE60DB9391054Aull;  // 2^64 / (2 pi)
  const unsigned bits = __float_as_uint(freq) & 0x7fffffffu;
  const int e = static_cast<int>(bits >> 23);
  const unsigned long long m = e ? (bits & 0x7fffffu) | 0x800000u : bits;
  const int shift = (e ? e : 1) - 150;  // |freq| = m 2^shift
  const unsigned long long hi = __umul64hi(m, kInv2Pi), lo = m * kInv2Pi;
  unsigned long long u;
  if (shift >= 0) u = shift < 64 ? lo << shift : 0;  // whole turns go
  else if (shift > -64) u = (lo >> -shift) | (hi << (64 + shift));
  else u = shift > -128 ? hi >> (-shift - 64) : 0;
  return freq < 0.f ? 0ull - u : u;
}
__device__ __forceinline__ void angle_of(int pos, unsigned long long turn, float* sin_, float* cos_) {
  const unsigned long long t = static_cast<unsigned long long>(static_cast<long long>(pos)) * turn;
  sincospif(static_cast<float>(static_cast<int>(t >> 32)) * 0x1p-31f, sin_, cos_);
}

// A pair's turn and axis; one that is not usable turns nothing, and is recorded.
struct Pair {
  unsigned long long turn;
  int axis;
};
__device__ __forceinline__ Pair pair_of(const RotateArgs& a, int i) {
  Pair p{0, 0};
  if (i >= a.rotary / 2) return p;
  const float f = a.freq[i];
  const int axis = a.axis ? a.axis[i] : 0;
  if (axis < 0 || axis >= a.axes || !(fabsf(f) < __builtin_huge_valf())) {
    atomicCAS(a.err, 0, 1);  // CB_ERR_INVALID_ARG
    return p;
  }
  p.turn = turn_of(f);
  p.axis = axis;
  return p;
}

// Any dims and strides: a warp per head of a token.
template <typename T>
__global__ void __launch_bounds__(32 * kWarps) rotate_rows_kernel(const RotateArgs a, long long rows) {
  __shared__ float y_s[kWarps][2 * kMaxPairs];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, all = a.v[0].heads + a.v[1].heads;
  float* y = y_s[warp];
  pdl_wait();
  pdl_launch_dependents();
  const Pair mine[2] = {pair_of(a, lane), pair_of(a, lane + 32)};
  for (long long r = static_cast<long long>(blockIdx.x) * kWarps + warp; r < rows; r += static_cast<long long>(gridDim.x) * kWarps) {
    const long long token = r / all;
    const int h = static_cast<int>(r - token * all), b = static_cast<int>(token / a.L), l = static_cast<int>(token - static_cast<long long>(b) * a.L);
    const RotateView& v = h < a.v[0].heads ? a.v[0] : a.v[1];
    const int head = h < a.v[0].heads ? h : h - a.v[0].heads;
    const T* x = static_cast<const T*>(v.x) + b * v.xs_b + l * v.xs_l + head * v.xs_h;
    T* out = static_cast<T*>(v.y) + b * v.ys_b + l * v.ys_l + head * v.ys_h;
    float e[4], sum = 0.f;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      e[c] = lane + 32 * c < a.dim ? to_f32(x[lane + 32 * c]) : 0.f;
      sum = fmaf(e[c], e[c], sum);
    }
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    const float inv = a.norm ? rsqrtf(sum / static_cast<float>(a.dim) + a.eps) : 1.f;
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int d = lane + 32 * c;
      if (d < a.dim) y[d] = a.norm ? e[c] * inv * (v.weight ? v.weight[d] : 1.f) : e[c];
    }
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int i = lane + 32 * c;
      if (i >= a.rotary / 2) break;
      float s, co;
      angle_of(a.pos[mine[c].axis * a.ps_a + b * a.ps_b + l], mine[c].turn, &s, &co);
      const int d1 = a.adjacent ? 2 * i : i, d2 = a.adjacent ? 2 * i + 1 : i + a.rotary / 2;
      const float y1 = y[d1], y2 = y[d2];
      out[d1] = from_f32<T>(y1 * co - y2 * s);
      out[d2] = from_f32<T>(y2 * co + y1 * s);
    }
    for (int d = a.rotary + lane; d < a.dim; d += 32) out[d] = from_f32<T>(y[d]);
  }
}

}  // namespace

cudaError_t launch_norm_rotate(const RotateArgs& a, bool bf16, bool vec, int sms, cudaStream_t s) {
  const long long rows = static_cast<long long>(a.B) * a.L * (a.v[0].heads + a.v[1].heads);
  const long long ctas = (rows + kWarps - 1) / kWarps, most = 16LL * sms;
  const dim3 grid(static_cast<unsigned>(ctas < most ? ctas : most)), block(32 * kWarps);
  return bf16 ? launch_pdl(rotate_rows_kernel<__nv_bfloat16>, grid, block, 0, s, a, rows)
              : launch_pdl(rotate_rows_kernel<float>, grid, block, 0, s, a, rows);
}

}  // namespace cb
