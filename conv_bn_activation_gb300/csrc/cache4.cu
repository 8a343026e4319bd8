// Tokens into the pages of a 4-bit cache and back (cb_cache4_append,
// cb_cache4_read).  Both are bound by HBM: 16 or 32 bits an element on one side
// and 4.5 on the other.
#include "cache4.cuh"
#include "launch_util.h"
#include "ptx.cuh"

namespace cb {

namespace {

constexpr int kWarps = 4;

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

unsigned grid_of(long long rows, int sms) {
  const long long ctas = (rows + kWarps - 1) / kWarps, most = 16LL * sms;
  return static_cast<unsigned>(ctas < most ? ctas : most);
}

}  // namespace

cudaError_t launch_cache4_append(const AppendArgs& a, bool bf16, bool vec, int sms, cudaStream_t s) {
  const long long rows = 2LL * a.B * a.T * a.H;
  return bf16 ? launch_pdl(cache4_append_rows_kernel<__nv_bfloat16>, dim3(grid_of(rows, sms)), dim3(32 * kWarps), 0, s, a, rows)
              : launch_pdl(cache4_append_rows_kernel<float>, dim3(grid_of(rows, sms)), dim3(32 * kWarps), 0, s, a, rows);
}

cudaError_t launch_cache4_read(const Read4Args& a, bool bf16, bool vec, int sms, cudaStream_t s) {
  const long long rows = 2LL * a.B * a.T * a.H;
  return bf16 ? launch_pdl(cache4_read_rows_kernel<__nv_bfloat16>, dim3(grid_of(rows, sms)), dim3(32 * kWarps), 0, s, a, rows)
              : launch_pdl(cache4_read_rows_kernel<float>, dim3(grid_of(rows, sms)), dim3(32 * kWarps), 0, s, a, rows);
}

}  // namespace cb
