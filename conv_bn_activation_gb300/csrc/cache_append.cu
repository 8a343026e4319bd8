// New tokens' keys and values into the pages of a cache (cb_cache_append).
//
// Pure movement, bound by HBM: each byte is read once and written once, in
// 16-byte pieces where the views allow it.  One CTA takes one token at a time:
// its page is looked up once, and its heads' keys, then values, are dealt
// piece by piece to the threads, so a warp moves 512 contiguous bytes of a
// packed row per access.
#include "internal.h"
#include "launch_util.h"
#include "ptx.cuh"

namespace cb {

namespace {

template <typename P>
__global__ void __launch_bounds__(128) cache_append_kernel(AppendArgs a, int elem_bytes, long long tokens) {
  pdl_wait();
  pdl_launch_dependents();
  const int per = static_cast<int>(sizeof(P)) / elem_bytes;  // elements per piece
  const int kp = a.dk / per, vp = a.dv / per, pieces = a.H * (kp + vp);
  for (long long w = blockIdx.x; w < tokens; w += gridDim.x) {
    const int b = static_cast<int>(w / a.T), t = static_cast<int>(w - static_cast<long long>(b) * a.T);
    if (a.count && t >= a.count[b]) continue;
    const long long at = static_cast<long long>(a.pos[b]) + t;
    const long long pg = at / a.cache.page_size;
    int page = -1;
    if (at >= 0 && pg < a.cache.max_pages) page = a.cache.table[b * a.cache.table_stride + pg];
    if (page < 0 || page >= a.cache.num_pages) {
      if (threadIdx.x == 0) atomicCAS(a.err, 0, 1);  // CB_ERR_INVALID_ARG
      continue;
    }
    const long long slot = at - pg * a.cache.page_size;
    const char* ks = static_cast<const char*>(a.k) + (b * a.ks_b + t * a.ks_l) * elem_bytes;
    const char* vs = static_cast<const char*>(a.v) + (b * a.vs_b + t * a.vs_l) * elem_bytes;
    char* kd = static_cast<char*>(a.cache.k) + (page * a.cache.ks_p + slot * a.cache.ks_t) * elem_bytes;
    char* vd = static_cast<char*>(a.cache.v) + (page * a.cache.vs_p + slot * a.cache.vs_t) * elem_bytes;
    for (int e = threadIdx.x; e < pieces; e += blockDim.x) {
      const bool is_v = e >= a.H * kp;
      const int x = is_v ? e - a.H * kp : e, n = is_v ? vp : kp;
      const int h = x / n, c = x - h * n;
      if (is_v)
        *reinterpret_cast<P*>(vd + h * a.cache.vs_h * elem_bytes + c * sizeof(P)) =
            *reinterpret_cast<const P*>(vs + h * a.vs_h * elem_bytes + c * sizeof(P));
      else
        *reinterpret_cast<P*>(kd + h * a.cache.ks_h * elem_bytes + c * sizeof(P)) =
            *reinterpret_cast<const P*>(ks + h * a.ks_h * elem_bytes + c * sizeof(P));
    }
  }
}

template <typename P>
cudaError_t launch_piece(const AppendArgs& a, int elem_bytes, int sms, cudaStream_t s) {
  const long long tokens = static_cast<long long>(a.B) * a.T;
  const long long grid = tokens < 16LL * sms ? tokens : 16LL * sms;
  return launch_pdl(cache_append_kernel<P>, dim3(static_cast<unsigned>(grid)), dim3(128), 0, s, a, elem_bytes, tokens);
}

}  // namespace

cudaError_t launch_cache_append(const AppendArgs& a, int elem_bytes, int piece, int sms, cudaStream_t s) {
  if (piece == 16) return launch_piece<uint4>(a, elem_bytes, sms, s);
  if (piece == 4) return launch_piece<uint32_t>(a, elem_bytes, sms, s);
  return launch_piece<uint16_t>(a, elem_bytes, sms, s);
}

}  // namespace cb
