// New tokens' keys and values into the pages of a cache (cb_cache_append).
//
// Pure movement, bound by HBM: each byte is read once and written once, in
// 16-byte pieces where the views allow it.  A warp takes 32 U pieces of one
// token at a time, always the same ones: which head and dims they are, and
// where in a token's row and in a page's slot, is worked out once per launch.
// All U reads of a lane are in flight before it looks the token's page up.
// 16 prompts of up to 2048 tokens, 8 heads of 128 (201 MB read and written):
// 33.7 us, 0.89 of the measured copy rate; with one read in flight per lane and
// a token per CTA 42.9.
#include "internal.h"
#include "launch_util.h"
#include "ptx.cuh"

namespace cb {

namespace {

constexpr int kWarps = 4;

// Each token is `chunks` units; the `warps` warps that work (a multiple of
// chunks) take units warp, warp + warps, ...
template <typename P, int U>
__global__ void __launch_bounds__(32 * kWarps)
cache_append_kernel(AppendArgs a, int elem_bytes, long long tokens, int chunks, int warps) {
  const int lane = threadIdx.x & 31, warp = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int per = static_cast<int>(sizeof(P)) / elem_bytes;  // elements per piece
  const int kp = a.dk / per, vp = a.dv / per, pieces = a.H * (kp + vp), first = warp % chunks * (32 * U) + lane;
  long long from[U], to[U];  // in bytes, from the token's row and the page's slot
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int e = min(first + 32 * u, pieces - 1);
    const bool is_v = e >= a.H * kp;
    const int x = is_v ? e - a.H * kp : e, n = is_v ? vp : kp, h = x / n, c = (x - h * n) * static_cast<int>(sizeof(P));
    from[u] = h * (is_v ? a.vs_h : a.ks_h) * elem_bytes + c;
    to[u] = h * (is_v ? a.cache.vs_h : a.cache.ks_h) * elem_bytes + c;
  }
  const int keys = a.H * kp;  // pieces before the values'
  pdl_launch_dependents();
  pdl_wait();
  if (warp >= warps) return;
  const long long step = warps / chunks, token = warp / chunks;
  const int step_b = static_cast<int>(step / a.T), step_t = static_cast<int>(step % a.T);
  int b = static_cast<int>(token / a.T), t = static_cast<int>(token % a.T);
  for (long long w = token; w < tokens; w += step, b += step_b, t += step_t) {
    if (t >= a.T) t -= a.T, ++b;
    if (a.count && t >= a.count[b]) continue;
    const char* ks = static_cast<const char*>(a.k) + (b * a.ks_b + t * a.ks_l) * elem_bytes;
    const char* vs = static_cast<const char*>(a.v) + (b * a.vs_b + t * a.vs_l) * elem_bytes;
    P v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (first + 32 * u < pieces) v[u] = *reinterpret_cast<const P*>((first + 32 * u < keys ? ks : vs) + from[u]);
    const long long at = static_cast<long long>(a.pos[b]) + t;
    const long long pg = at / a.cache.page_size;
    int page = -1;
    if (at >= 0 && pg < a.cache.max_pages) page = a.cache.table[b * a.cache.table_stride + pg];
    if (page < 0 || page >= a.cache.num_pages) {
      if (lane == 0) atomicCAS(a.err, 0, 1);  // CB_ERR_INVALID_ARG
      continue;
    }
    const long long slot = at - pg * a.cache.page_size;
    char* kd = static_cast<char*>(a.cache.k) + (page * a.cache.ks_p + slot * a.cache.ks_t) * elem_bytes;
    char* vd = static_cast<char*>(a.cache.v) + (page * a.cache.vs_p + slot * a.cache.vs_t) * elem_bytes;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (first + 32 * u < pieces) *reinterpret_cast<P*>((first + 32 * u < keys ? kd : vd) + to[u]) = v[u];
  }
}

template <typename P, int U>
cudaError_t launch_units(const AppendArgs& a, int elem_bytes, long long tokens, int pieces, int sms, cudaStream_t s) {
  const int chunks = (pieces + 32 * U - 1) / (32 * U);
  const long long units = tokens * chunks, most = 4LL * sms * kWarps;
  const long long warps = units < most ? units : (most < chunks ? chunks : most / chunks * chunks);
  return launch_pdl(cache_append_kernel<P, U>, dim3(static_cast<unsigned>((warps + kWarps - 1) / kWarps)), dim3(32 * kWarps), 0, s, a,
                    elem_bytes, tokens, chunks, static_cast<int>(warps));
}

template <typename P>
cudaError_t launch_piece(const AppendArgs& a, int elem_bytes, int sms, cudaStream_t s) {
  const long long tokens = static_cast<long long>(a.B) * a.T;
  const int pieces = a.H * static_cast<int>((a.dk + a.dv) * elem_bytes / sizeof(P));
  // A CTA's worth of pieces per SM or fewer: one to a lane (64 tokens of 8 heads of 128 and 128 bf16:
  // 1.74 us, with eight 1.93); more: eight (385 tokens of 4 heads of 32 and 64 fp32: 1.81, with one 1.90).
  if (tokens * pieces <= 32LL * kWarps * sms) return launch_units<P, 1>(a, elem_bytes, tokens, pieces, sms, s);
  return launch_units<P, 8>(a, elem_bytes, tokens, pieces, sms, s);
}

}  // namespace

cudaError_t launch_cache_append(const AppendArgs& a, int elem_bytes, int piece, int sms, cudaStream_t s) {
  if (piece == 16) return launch_piece<uint4>(a, elem_bytes, sms, s);
  if (piece == 4) return launch_piece<uint32_t>(a, elem_bytes, sms, s);
  return launch_piece<uint16_t>(a, elem_bytes, sms, s);
}

}  // namespace cb
