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

#include <initializer_list>

#include "attention_common.cuh"
#include "launch_util.h"
#include "ptx.cuh"

namespace cb {

namespace {

constexpr int kWarps = 4;
constexpr int kMaxPairs = 64;
constexpr int kPiecesCtas = 5, kDepth = 3;  // resident CTAs an SM; groups copied ahead

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

template <int BYTES>
__device__ __forceinline__ void copy_ahead(void* dst, const void* src) {
  if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(dst)), "l"(src), "n"(BYTES) : "memory");
}

// E elements of a row, and as pairs of fp32.
template <typename T, int E>
struct alignas(E * sizeof(T)) Piece {
  static constexpr int kBytes = E * static_cast<int>(sizeof(T)), kWords = kBytes / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void get(f2* x) const {
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      if constexpr (sizeof(T) == 4) x[i] = pack2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
      else x[i] = pack2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
  }
  __device__ __forceinline__ void set(const f2* x) {
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      float lo, hi;
      unpack2(x[i], lo, hi);
      if constexpr (sizeof(T) == 4) {
        w[2 * i] = __float_as_uint(lo), w[2 * i + 1] = __float_as_uint(hi);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
  }
};

// Rows of whole pieces of E elements, 16 bytes where dims and strides allow them,
// else 8 or 4, and pairs in whole pieces.  Bound by HBM.  `width`
// lanes (a power of two) share a head, each with two pieces of it: the halves of
// the same pairs, or, adjacent pairs, any two; what does not turn is split in
// halves too and turns by 0.  A warp works on queries or on keys: 32 / width heads
// of a token at a time, every `parts`-th such group of its heads, then the next
// token's.  Each lane copies its pieces ahead through a ring of its own in shared
// memory: kDepth groups, where two in registers left the memory waiting (84 us
// for 16384 tokens of 40 heads of 128, so 58).  A token's angles, two to a lane,
// go through shared memory to the lanes that need them, times the weights.
struct Split {  // of the grid's warps: the first `warps` of a view's kind, `parts` to a token
  unsigned warps[2], parts[2];
};
template <typename T, int E, bool ADJ>
__global__ void __launch_bounds__(32 * kWarps, kPiecesCtas) rotate_pieces_kernel(const RotateArgs a, const int width, const Split split) {
  constexpr int H = E / 2;  // pairs of fp32 in a piece
  using Part = Piece<T, E>;
  __shared__ __align__(16) Part ring_s[kWarps][kDepth][2][32];
  __shared__ int pos_s[kWarps][kDepth][2][32];
  __shared__ __align__(16) float weight_s[2][2 * kMaxPairs];
  __shared__ __align__(16) float cos_s[kWarps][kMaxPairs], sin_s[kWarps][kMaxPairs];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane & (width - 1), slot = lane / width, slots = 32 / width;
  const int half = a.rotary / 2, turning = a.rotary / (2 * E);  // lanes of a head that hold turning halves
  int p0 = sub * E, p1 = p0 + a.dim / 2;
  if (!ADJ) {
    if (sub < turning) p1 = p0 + half;
    else p0 = a.rotary + (sub - turning) * E, p1 = p0 + (a.dim - a.rotary) / 2;
  }
  unsigned unit = blockIdx.x * kWarps + warp;
  const bool is_k = unit >= split.warps[0];
  if (is_k) unit -= split.warps[0];
  const RotateView& v = a.v[is_k];
  const unsigned parts = max(split.parts[is_k], 1u), part = unit % parts, step = split.warps[is_k] / parts;
  const unsigned heads = v.heads, advance = parts * slots, first = part * slots + slot;
  const unsigned tokens = static_cast<unsigned>(a.B) * static_cast<unsigned>(a.L);
  const bool mine = sub < a.dim / (2 * E), still = a.rotary < a.dim;  // still: some dims do not turn
  const float inv_dim = 1.f / static_cast<float>(a.dim);
  const unsigned xs_h = static_cast<unsigned>(v.xs_h), ys_h = static_cast<unsigned>(v.ys_h);
  float* const cos_ = cos_s[warp];
  float* const sin_ = sin_s[warp];
  pdl_wait();
  pdl_launch_dependents();
  const Pair pair[2] = {pair_of(a, lane), pair_of(a, lane + 32)};
  const float* const weights = weight_s[is_k];

  struct Place {
    unsigned token, head;  // this lane's; a token's last group may have none for it
  };
  // Where the next rows to fetch lie, and where the next results go.
  const T* x_at = nullptr;
  T* y_at = nullptr;
  auto fetch = [&](const Place& r, int at) {
    if (r.token < tokens) {
      if (r.head == first) {  // a new token
        const unsigned b = r.token / static_cast<unsigned>(a.L), l = r.token - b * a.L;
        x_at = static_cast<const T*>(v.x) + b * v.xs_b + l * v.xs_l + p0;
        const int* pos = a.pos + b * a.ps_b + l;
#pragma unroll
        for (int c = 0; c < 2; ++c)
          if (lane + 32 * c < half) copy_ahead<4>(&pos_s[warp][at][c][lane], pos + pair[c].axis * a.ps_a);
      }
      if (mine && r.head < heads) {
        const T* x = x_at + static_cast<unsigned long long>(r.head) * xs_h;
        copy_ahead<Part::kBytes>(&ring_s[warp][at][0][lane], x);
        copy_ahead<Part::kBytes>(&ring_s[warp][at][1][lane], x + (p1 - p0));
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto next = [&](Place& r) {
    r.head += advance;
    if (r.head - slot >= heads) r.head = first, r.token += step;
  };
  // Of this lane's pairs, y = inv x (first: with a large weight a product could leave fp32's range): z1 = y1 (w1 cos) - y2
  // (w2 sin), z2 = y2 (w2 cos) + y1 (w1 sin); adjacent pairs as (z1, z2) = (y1, y2) (w1 cos, w2 cos) + (y2, y1) (-w2 sin, w1 sin).
  f2 c1[H], c2[H], s1[H], s2[H];
  auto work = [&](const Place& r, int at) {
    if (r.head == first) {
      const unsigned b = r.token / static_cast<unsigned>(a.L), l = r.token - b * a.L;
      y_at = static_cast<T*>(v.y) + b * v.ys_b + l * v.ys_l + p0;
      __syncwarp();
#pragma unroll
      for (int c = 0; c < 2; ++c)
        if (lane + 32 * c < half) angle_of(pos_s[warp][at][c][lane], pair[c].turn, &sin_[lane + 32 * c], &cos_[lane + 32 * c]);
      __syncwarp();
      auto weight = [&](int d) { return mine ? weights[d] : 0.f; };
#pragma unroll
      for (int i = 0; i < H; ++i) {
        if constexpr (ADJ) {  // pairs i of either piece
          const float ca = cos_[p0 / 2 + i], sa = sin_[p0 / 2 + i], cb = cos_[p1 / 2 + i], sb = sin_[p1 / 2 + i];
          const float wa = weight(p0 + 2 * i), wb = weight(p0 + 2 * i + 1), wc = weight(p1 + 2 * i), wd = weight(p1 + 2 * i + 1);
          c1[i] = pack2(wa * ca, wb * ca), s1[i] = pack2(-wb * sa, wa * sa);
          c2[i] = pack2(wc * cb, wd * cb), s2[i] = pack2(-wd * sb, wc * sb);
        } else {  // pairs 2 i and 2 i + 1, whose halves the pieces are
          const float2 co = *reinterpret_cast<const float2*>(cos_ + sub * E + 2 * i), si = *reinterpret_cast<const float2*>(sin_ + sub * E + 2 * i);
          const float wa = weight(p0 + 2 * i), wb = weight(p0 + 2 * i + 1), wc = weight(p1 + 2 * i), wd = weight(p1 + 2 * i + 1);
          c1[i] = pack2(wa * co.x, wb * co.y), s1[i] = pack2(wa * si.x, wb * si.y);
          c2[i] = pack2(wc * co.x, wd * co.y), s2[i] = pack2(-wc * si.x, -wd * si.y);
        }
      }
    }
    f2 x[E];  // piece 0, piece 1
    ring_s[warp][at][0][lane].get(x), ring_s[warp][at][1][lane].get(x + H);
    f2 inv = pack2(1.f, 1.f);
    if (a.norm) {
      f2 sums = mul2(x[0], x[0]);
#pragma unroll
      for (int i = 1; i < E; ++i) sums = fma2(x[i], x[i], sums);
      float lo, hi;
      unpack2(sums, lo, hi);
      float sum = lo + hi;
      for (int o = width / 2; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
      const float f = rsqrtf(fmaf(sum, inv_dim, a.eps));
      inv = pack2(f, f);
    }
    // What does not turn takes nothing from the other dim of its pair, an infinity or NaN neither.
    auto other = [&](f2 y, int i) { return still && i >= half ? pack2(0.f, 0.f) : y; };
#pragma unroll
    for (int i = 0; i < H; ++i) {
      const f2 y1 = mul2(x[i], inv), y2 = mul2(x[H + i], inv);
      if constexpr (ADJ) {
        float u, w;
        unpack2(y1, u, w);
        x[i] = fma2(other(pack2(w, u), p0 / 2 + i), s1[i], mul2(y1, c1[i]));
        unpack2(y2, u, w);
        x[H + i] = fma2(other(pack2(w, u), p1 / 2 + i), s2[i], mul2(y2, c2[i]));
      } else {
        x[i] = fma2(other(y2, sub * E), s2[i], mul2(y1, c1[i]));
        x[H + i] = fma2(other(y1, sub * E), s1[i], mul2(y2, c2[i]));
      }
    }
    if (mine && r.head < heads) {
      T* y = y_at + static_cast<unsigned long long>(r.head) * ys_h;
      Part out;
      out.set(x);
      *reinterpret_cast<Part*>(y) = out;
      out.set(x + H);
      *reinterpret_cast<Part*>(y + (p1 - p0)) = out;
    }
  };
  if (!mine)  // what is never copied adds nothing to a norm
    for (int at = 0; at < kDepth; ++at) ring_s[warp][at][0][lane] = ring_s[warp][at][1][lane] = Part{};
  Place ahead{unit < split.warps[is_k] ? unit / parts : tokens, first}, now = ahead;
#pragma unroll
  for (int at = 0; at < kDepth - 1; ++at) fetch(ahead, at), next(ahead);
  cos_[lane] = cos_[lane + 32] = 1.f, sin_[lane] = sin_[lane + 32] = 0.f;  // what does not turn
  for (int d = threadIdx.x; d < 2 * a.dim; d += 32 * kWarps) {
    const float* w = a.v[d >= a.dim].weight;
    weight_s[d >= a.dim][d % a.dim] = w ? w[d % a.dim] : 1.f;
  }
  __syncthreads();
  int at = 0;
  while (now.token < tokens) {
    fetch(ahead, at == 0 ? kDepth - 1 : at - 1);
    next(ahead);
    asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
    work(now, at);
    next(now);
    at = at + 1 == kDepth ? 0 : at + 1;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

template <typename T, int E>
cudaError_t launch_pieces(const RotateArgs& a, int sms, cudaStream_t s) {
  int width = 1;
  while (width * 2 * E < a.dim) width *= 2;
  const int slots = 32 / width;
  const long long tokens = static_cast<long long>(a.B) * a.L;
  const long long groups[2] = {(a.v[0].heads + slots - 1) / slots, (a.v[1].heads + slots - 1) / slots};
  // The resident warps are dealt to queries and keys by their work: their groups and, per token, its angles and
  // weights, which cost about as much as a group.  A token's heads go to as many warps as that leaves idle.
  const long long most = static_cast<long long>(kPiecesCtas) * kWarps * sms, work[2] = {groups[0] + 1, groups[1] ? groups[1] + 1 : 0};
  Split split{};
  for (int v = 0; v < 2; ++v) {
    if (!groups[v]) continue;
    long long warps = most * work[v] / (work[0] + work[1]);
    if (warps < 1) warps = 1;
    long long parts = warps / tokens;
    parts = parts < 1 ? 1 : parts > groups[v] ? groups[v] : parts;
    if (warps > tokens * parts) warps = tokens * parts;
    split.parts[v] = static_cast<unsigned>(parts);
    split.warps[v] = static_cast<unsigned>((warps + parts - 1) / parts * parts);
  }
  const unsigned ctas = (split.warps[0] + split.warps[1] + kWarps - 1) / kWarps;
  auto* kernel = a.adjacent ? rotate_pieces_kernel<T, E, true> : rotate_pieces_kernel<T, E, false>;
  return launch_pdl(kernel, dim3(ctas), dim3(32 * kWarps), 0, s, a, width, split);
}

// Whether rows are pieces of E elements, pairs lie in whole ones, and a head's offset in its token fits 32 bits.
template <typename T, int E>
bool pieces(const RotateArgs& a) {
  if (a.dim % (2 * E) != 0 || (!a.adjacent && a.rotary % (2 * E) != 0)) return false;
  for (const RotateView& v : a.v) {
    if (!v.heads) continue;
    if ((reinterpret_cast<uintptr_t>(v.x) | reinterpret_cast<uintptr_t>(v.y)) % (E * sizeof(T)) != 0) return false;
    for (const long long stride : {v.xs_b, v.xs_l, v.xs_h, v.ys_b, v.ys_l, v.ys_h})
      if (stride % E != 0) return false;
    if (v.xs_h >= (1LL << 31) || v.ys_h >= (1LL << 31)) return false;
  }
  return true;
}

}  // namespace

cudaError_t launch_norm_rotate(const RotateArgs& a, bool bf16, int sms, cudaStream_t s) {
  if (bf16) {
    if (pieces<__nv_bfloat16, 8>(a)) return launch_pieces<__nv_bfloat16, 8>(a, sms, s);
    if (pieces<__nv_bfloat16, 4>(a)) return launch_pieces<__nv_bfloat16, 4>(a, sms, s);
    if (pieces<__nv_bfloat16, 2>(a)) return launch_pieces<__nv_bfloat16, 2>(a, sms, s);
  } else {
    if (pieces<float, 4>(a)) return launch_pieces<float, 4>(a, sms, s);
    if (pieces<float, 2>(a)) return launch_pieces<float, 2>(a, sms, s);
  }
  const long long rows = static_cast<long long>(a.B) * a.L * (a.v[0].heads + a.v[1].heads);
  const long long ctas = (rows + kWarps - 1) / kWarps, most = 16LL * sms;
  const dim3 grid(static_cast<unsigned>(ctas < most ? ctas : most)), block(32 * kWarps);
  return bf16 ? launch_pdl(rotate_rows_kernel<__nv_bfloat16>, grid, block, 0, s, a, rows)
              : launch_pdl(rotate_rows_kernel<float>, grid, block, 0, s, a, rows);
}

}  // namespace cb
