// Tokens into the pages of a 4-bit cache and back (cb_cache4_append,
// cb_cache4_read).  Both are bound by HBM: 16 or 32 bits an element on one side
// and 4.5 on the other.
//
// Rows of whole words (dims that are multiples of 8) and 16-byte pieces: a lane
// takes eight dims of a row, a word of codes, so four lanes share a group and its
// scale (the last one's may have nothing).  A token's words of all heads, keys then values, lie side by side over
// the lanes; which head and dims a lane's words are, and where they lie in a
// token's row and a page's slot, is worked out once per launch, as in
// cache_append.cu.  The reads of all a lane's words are in flight before it
// looks the token's page up.  16 prompts of up to 2048 tokens, 8 heads of 128
// bf16: stored in 44 us, of 19 at the copy rate (bound by instructions: 0.70 of the
// issue slots, about 100 for a word and the rest a token's addresses), 16384 such
// tokens read in 18.4, of 12.7 (15.6 where the L2 still holds the codes).  One warp
// per head (the kernels for other rows) took 4 to 6 times as long.  A lane's words
// are of one token: with few key heads most lanes have none, and cases for many
// words go far from their floor (32 maps of 400 tokens, 2 heads of 32, fp32: read
// in 10.7 us, of 1.1).
#include "cache4.cuh"
#include "launch_util.h"
#include "ptx.cuh"

namespace cb {

namespace {

constexpr int kWarps = 4;
// CTAs for each SM at most, by heads of 128 dims alone, 4 and 8 of them, on codes that the L2 may hold.  Counts leave some
// with little: more than the SM holds (stored and read as above, 6: 73 us, 8: 77, 12: 69, 16: 67.5, 24: 71).  Without counts all have the same: what it holds at once when tokens are read (16 k of them,
// 6: 15.7 us, 8: 18.3, 16: 17.7), twice that when they are stored (16 k of 4 heads, 6: 13.5, 12: 14.1, 16: 14.8; 32 k of 8,
// 6: 52, 12: 47, 16: 49).
constexpr int kReadCtas = 6;
constexpr long long kCountedCtas = 16, kStoreCtas = 2 * kReadCtas;

// A warp per head of a token's keys or values: a lane per dim of a group.
template <typename T>
__global__ void __launch_bounds__(32 * kWarps) cache4_append_rows_kernel(const AppendArgs a, long long rows) {
  const int lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  for (long long r = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5); r < rows;
       r += static_cast<long long>(gridDim.x) * kWarps) {
    const long long token = r / (2 * a.H);
    const int part = static_cast<int>(r - token * (2 * a.H)), h = part >> 1;
    const bool is_v = part & 1;
    const int b = static_cast<int>(token / a.T), t = static_cast<int>(token - static_cast<long long>(b) * a.T);
    if (a.count && t >= a.count[b]) continue;
    int slot = 0;
    const int page = cache_page(a.cache, a.err, b, static_cast<long long>(a.pos[b]) + t, &slot);
    if (page < 0) continue;
    const int dim = is_v ? a.dv : a.dk;
    const T* x = is_v ? static_cast<const T*>(a.v) + b * a.vs_b + t * a.vs_l + h * a.vs_h
                      : static_cast<const T*>(a.k) + b * a.ks_b + t * a.ks_l + h * a.ks_h;
    uint8_t* codes = const_cast<uint8_t*>(is_v ? value_codes4(a.cache, page, slot, h) : key_codes4(a.cache, page, slot, h));
    uint16_t* scales = const_cast<uint16_t*>(is_v ? value_scales4(a.cache, page, slot, h) : key_scales4(a.cache, page, slot, h));
    for (int g = 0; g < scales4(dim); ++g) {
      const int d = g * kGroup4 + lane;
      const float e = d < dim ? to_f32(x[d]) : 0.f;
      const unsigned bits = scale4_bits(__reduce_max_sync(~0u, __float_as_uint(e) & 0x7fffffffu));
      const unsigned n = Coder4(bits).nibble(e), next = __shfl_down_sync(~0u, n, 1);
      if (d < dim && !(lane & 1)) codes[d >> 1] = static_cast<uint8_t>(n | (next << 4));
      if (lane == 0) scales[g] = static_cast<uint16_t>(bits);
    }
  }
}

// A warp per head of a token's keys or values.
template <typename T>
__global__ void __launch_bounds__(32 * kWarps) cache4_read_rows_kernel(const Read4Args a, long long rows) {
  const int lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  for (long long r = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5); r < rows;
       r += static_cast<long long>(gridDim.x) * kWarps) {
    const long long token = r / (2 * a.H);
    const int part = static_cast<int>(r - token * (2 * a.H)), h = part >> 1;
    const bool is_v = part & 1;
    const int b = static_cast<int>(token / a.T), t = static_cast<int>(token - static_cast<long long>(b) * a.T);
    if (a.count && t >= a.count[b]) continue;
    int slot = 0;
    const int page = cache_page(a.cache, a.err, b, (a.first ? static_cast<long long>(a.first[b]) : 0) + t, &slot);
    const int dim = is_v ? a.dv : a.dk;
    T* y = is_v ? static_cast<T*>(a.v) + b * a.vs_b + t * a.vs_l + h * a.vs_h : static_cast<T*>(a.k) + b * a.ks_b + t * a.ks_l + h * a.ks_h;
    const uint8_t* codes = is_v ? value_codes4(a.cache, page, slot, h) : key_codes4(a.cache, page, slot, h);
    const uint16_t* scales = is_v ? value_scales4(a.cache, page, slot, h) : key_scales4(a.cache, page, slot, h);
    for (int d = lane; d < dim; d += 32) y[d] = from_f32<T>(page < 0 ? 0.f : value4(codes, scales, d));
  }
}

// Eight elements of a row.
template <typename T>
struct Eight {
  uint4 w[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  // The largest of their bits without sign, as fp32's.
  __device__ __forceinline__ unsigned top() const {
    if constexpr (sizeof(T) == 4) {
      unsigned m = 0;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        m = max(max(m, max(w[i].x & 0x7fffffffu, w[i].y & 0x7fffffffu)), max(w[i].z & 0x7fffffffu, w[i].w & 0x7fffffffu));
      return m;
    } else {
      const unsigned m = max2(max2(w[0].x & 0x7fff7fffu, w[0].y & 0x7fff7fffu), max2(w[0].z & 0x7fff7fffu, w[0].w & 0x7fff7fffu));
      return max(m & 0xffff0000u, m << 16);
    }
  }
  static __device__ __forceinline__ unsigned max2(unsigned a, unsigned b) {
    unsigned m;
    asm("max.s16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
    return m;
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    if constexpr (sizeof(T) == 4) {
      unpack16<T>(w[0], *reinterpret_cast<float(*)[4]>(x));
      unpack16<T>(w[1], *reinterpret_cast<float(*)[4]>(x + 4));
    } else {
      unpack16<T>(w[0], x);
    }
  }
};

// Where a lane's words lie: elements from the token's row of keys or values,
// bytes from the slot's row of their codes, elements from that of their scales.
struct Word {
  bool is_v, real, writes;  // real: there is such a word, with such dims; writes: the lane that stores the group's scale
  int from, to, scale, group;
};
__device__ __forceinline__ int words4(int dim) { return (dim + kGroup4 - 1) / kGroup4 * 4; }
__device__ __forceinline__ Word word_of(int at, int words, int dk, int dv, int heads, long long ks_h, long long vs_h, const PagedArgs& c) {
  const int kw = words4(dk), vw = words4(dv), keys = heads * kw, e = min(at, words - 1);
  Word w;
  w.is_v = e >= keys;
  const int x = w.is_v ? e - keys : e, n = w.is_v ? vw : kw, h = x / n, i = x - h * n;
  w.from = static_cast<int>(h * (w.is_v ? vs_h : ks_h)) + 8 * i;
  w.to = static_cast<int>(h * (w.is_v ? c.vs_h : c.ks_h)) + 4 * i;
  w.group = i / 4;
  w.scale = static_cast<int>(h * (w.is_v ? c.vx_h : c.kx_h)) + w.group;
  w.real = at < words && 8 * i < (w.is_v ? dv : dk);
  w.writes = at < words && i % 4 == 0;
  return w;
}

// The token that a unit of a launch is about.
struct Walk {
  long long token, step, tokens;
  int b, t, step_b, step_t, T;
  __device__ __forceinline__ Walk(int warp, int warps, int chunks, int T_, long long tokens_) : T(T_) {
    step = warps / chunks, token = warp / chunks, tokens = tokens_;
    step_b = static_cast<int>(step / T), step_t = static_cast<int>(step - static_cast<long long>(step_b) * T);
    b = static_cast<int>(token / T), t = static_cast<int>(token - static_cast<long long>(b) * T);
  }
  __device__ __forceinline__ bool here() const { return token < tokens; }
  __device__ __forceinline__ void next() {
    token += step, b += step_b, t += step_t;
    if (t >= T) t -= T, ++b;
  }
};

template <typename T, int U>
__global__ void __launch_bounds__(32 * kWarps) cache4_append_kernel(const AppendArgs a, long long tokens, int chunks, int warps) {
  const int lane = threadIdx.x & 31, warp = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int words = a.H * (words4(a.dk) + words4(a.dv)), first = warp % chunks * (32 * U) + lane;
  Word w[U];
#pragma unroll
  for (int u = 0; u < U; ++u) w[u] = word_of(first + 32 * u, words, a.dk, a.dv, a.H, a.ks_h, a.vs_h, a.cache);
  const int last_k = words4(a.dk) / 4 - 1, last_v = words4(a.dv) / 4 - 1;  // groups; behind an even one a scale of zero
  pdl_wait();
  pdl_launch_dependents();
  if (warp >= warps) return;
  for (Walk at(warp, warps, chunks, a.T, tokens); at.here(); at.next()) {
    const int b = at.b, t = at.t;
    if (a.count && t >= a.count[b]) continue;
    const T* ks = static_cast<const T*>(a.k) + b * a.ks_b + t * a.ks_l;
    const T* vs = static_cast<const T*>(a.v) + b * a.vs_b + t * a.vs_l;
    Eight<T> x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      x[u] = {};
      if (w[u].real) x[u].load((w[u].is_v ? vs : ks) + w[u].from);
    }
    int slot = 0;
    const long long page = cache_page(a.cache, a.err, b, static_cast<long long>(a.pos[b]) + t, &slot);
    if (page < 0) continue;
    uint8_t* kd = const_cast<uint8_t*>(key_codes4(a.cache, page, slot, 0));
    uint8_t* vd = const_cast<uint8_t*>(value_codes4(a.cache, page, slot, 0));
    uint16_t* kx = const_cast<uint16_t*>(key_scales4(a.cache, page, slot, 0));
    uint16_t* vx = const_cast<uint16_t*>(value_scales4(a.cache, page, slot, 0));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float f[8];
      x[u].get(f);
      unsigned top = x[u].top();
      top = max(top, __shfl_xor_sync(~0u, top, 1));
      top = max(top, __shfl_xor_sync(~0u, top, 2));
      const unsigned bits = scale4_bits(top);
      const uint32_t code = Coder4(bits).word<sizeof(T) == 2>(f);
      if (w[u].real) *reinterpret_cast<uint32_t*>((w[u].is_v ? vd : kd) + w[u].to) = code;
      if (w[u].writes) {
        uint16_t* s = (w[u].is_v ? vx : kx) + w[u].scale;
        s[0] = static_cast<uint16_t>(bits);
        if (w[u].group % 2 == 0 && w[u].group == (w[u].is_v ? last_v : last_k)) s[1] = 0;
      }
    }
  }
}

template <typename T, int U>
__global__ void __launch_bounds__(32 * kWarps, kReadCtas) cache4_read_kernel(const Read4Args a, long long tokens, int chunks,
                                                                             int warps) {
  const int lane = threadIdx.x & 31, warp = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int words = a.H * (words4(a.dk) + words4(a.dv)), first = warp % chunks * (32 * U) + lane;
  Word w[U];
#pragma unroll
  for (int u = 0; u < U; ++u) w[u] = word_of(first + 32 * u, words, a.dk, a.dv, a.H, a.ks_h, a.vs_h, a.cache);
  pdl_wait();
  pdl_launch_dependents();
  if (warp >= warps) return;
  for (Walk at(warp, warps, chunks, a.T, tokens); at.here(); at.next()) {
    const int b = at.b, t = at.t;
    if (a.count && t >= a.count[b]) continue;
    int slot = 0;
    const long long page = cache_page(a.cache, a.err, b, (a.first ? static_cast<long long>(a.first[b]) : 0) + t, &slot);
    const uint8_t* ks = key_codes4(a.cache, page, slot, 0);
    const uint8_t* vs = value_codes4(a.cache, page, slot, 0);
    const uint16_t* kx = key_scales4(a.cache, page, slot, 0);
    const uint16_t* vx = value_scales4(a.cache, page, slot, 0);
    uint32_t code[U];
    unsigned scale[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      code[u] = 0x88888888u, scale[u] = 0;  // a token that has no page reads as zeros
      if (page >= 0 && w[u].real) {
        code[u] = *reinterpret_cast<const uint32_t*>((w[u].is_v ? vs : ks) + w[u].to);
        scale[u] = ((w[u].is_v ? vx : kx) + w[u].scale)[0];
      }
    }
    T* kd = static_cast<T*>(a.k) + b * a.ks_b + t * a.ks_l;
    T* vd = static_cast<T*>(a.v) + b * a.vs_b + t * a.vs_l;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!w[u].real) continue;
      uint4* y = reinterpret_cast<uint4*>((w[u].is_v ? vd : kd) + w[u].from);
      if constexpr (sizeof(T) == 4) {
        const float s = bf16_value(scale[u]);
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)  // 2^23 + (c + 8), less 2^23 + 8
          f[i] = (__uint_as_float(((code[u] >> (4 * i)) & 15u) | 0x4b000000u) - 8388616.f) * s;
        y[0] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
        y[1] = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
      } else {
        // Dims i and i + 4 as bf16: 128 + (c + 8), less 136, times s: one rounding, the product's.
        const uint32_t ss = scale[u] | (scale[u] << 16), base = 0xc308c308u;
        uint32_t p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t n = ((code[u] >> (4 * i)) & 0x000f000fu) | 0x43004300u;
          const __nv_bfloat162 c = __hadd2(*reinterpret_cast<const __nv_bfloat162*>(&n), *reinterpret_cast<const __nv_bfloat162*>(&base));
          const __nv_bfloat162 v = __hmul2(c, *reinterpret_cast<const __nv_bfloat162*>(&ss));
          p[i] = *reinterpret_cast<const uint32_t*>(&v);
        }
        y[0] = make_uint4(__byte_perm(p[0], p[1], 0x5410), __byte_perm(p[2], p[3], 0x5410), __byte_perm(p[0], p[1], 0x7632),
                          __byte_perm(p[2], p[3], 0x7632));
      }
    }
  }
}

template <typename T, int U, class Args, class Kernel>
cudaError_t launch_words(Kernel kernel, const Args& a, long long ctas, int sms, cudaStream_t s) {
  const long long tokens = static_cast<long long>(a.B) * a.T;
  const int words = a.H * 4 * ((a.dk + kGroup4 - 1) / kGroup4 + (a.dv + kGroup4 - 1) / kGroup4), chunks = (words + 32 * U - 1) / (32 * U);
  const long long units = tokens * chunks, most = (U == 1 || a.count ? kCountedCtas : ctas) * kWarps * sms;
  const long long warps = units < most ? units : (most < chunks ? chunks : most / chunks * chunks);
  return launch_pdl(kernel, dim3(static_cast<unsigned>((warps + kWarps - 1) / kWarps)), dim3(32 * kWarps), 0, s, a, tokens, chunks,
                    static_cast<int>(warps));
}

// Eight CTAs' worth of words per SM or fewer: one to a lane, so that a token's heads spread over the GPU; more: four to be
// stored (two 73 us, eight 73, four 67), eight to be read (16 CTAs: two 23 us, four 17.6, eight 16.9); measured with 8
// heads of 128.
template <class Args>
bool few_words(const Args& a, int sms) {
  return static_cast<long long>(a.B) * a.T * a.H * ((a.dk + a.dv) / 8) <= 32LL * kWarps * 8 * sms;
}

unsigned grid_of(long long rows, int sms) {
  const long long ctas = (rows + kWarps - 1) / kWarps, most = 16LL * sms;
  return static_cast<unsigned>(ctas < most ? ctas : most);
}

}  // namespace

cudaError_t launch_cache4_append(const AppendArgs& a, bool bf16, bool vec, int sms, cudaStream_t s) {
  if (vec) {
    if (few_words(a, sms))
      return bf16 ? launch_words<__nv_bfloat16, 1>(cache4_append_kernel<__nv_bfloat16, 1>, a, kStoreCtas, sms, s)
                  : launch_words<float, 1>(cache4_append_kernel<float, 1>, a, kStoreCtas, sms, s);
    return bf16 ? launch_words<__nv_bfloat16, 4>(cache4_append_kernel<__nv_bfloat16, 4>, a, kStoreCtas, sms, s)
                : launch_words<float, 4>(cache4_append_kernel<float, 4>, a, kStoreCtas, sms, s);
  }
  const long long rows = 2LL * a.B * a.T * a.H;
  return bf16 ? launch_pdl(cache4_append_rows_kernel<__nv_bfloat16>, dim3(grid_of(rows, sms)), dim3(32 * kWarps), 0, s, a, rows)
              : launch_pdl(cache4_append_rows_kernel<float>, dim3(grid_of(rows, sms)), dim3(32 * kWarps), 0, s, a, rows);
}

cudaError_t launch_cache4_read(const Read4Args& a, bool bf16, bool vec, int sms, cudaStream_t s) {
  if (vec) {
    if (few_words(a, sms))
      return bf16 ? launch_words<__nv_bfloat16, 1>(cache4_read_kernel<__nv_bfloat16, 1>, a, kReadCtas, sms, s)
                  : launch_words<float, 1>(cache4_read_kernel<float, 1>, a, kReadCtas, sms, s);
    return bf16 ? launch_words<__nv_bfloat16, 8>(cache4_read_kernel<__nv_bfloat16, 8>, a, kReadCtas, sms, s)
                : launch_words<float, 8>(cache4_read_kernel<float, 8>, a, kReadCtas, sms, s);
  }
  const long long rows = 2LL * a.B * a.T * a.H;
  return bf16 ? launch_pdl(cache4_read_rows_kernel<__nv_bfloat16>, dim3(grid_of(rows, sms)), dim3(32 * kWarps), 0, s, a, rows)
              : launch_pdl(cache4_read_rows_kernel<float>, dim3(grid_of(rows, sms)), dim3(32 * kWarps), 0, s, a, rows);
}

}  // namespace cb
