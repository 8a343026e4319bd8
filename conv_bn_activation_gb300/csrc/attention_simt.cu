// Attention in fp32 arithmetic on the CUDA cores: fp32 views, and bf16 views
// that the tensor-core kernel cannot address (attention_tc.cu).
//
// One CTA owns BM queries of one head and walks the visible keys in tiles of
// 64 with the running maximum m and sum l of the softmax: for each tile
//   x = log2(e) * score, m' = max(m, max x), p = 2^(x - m'),
//   o = o * 2^(m - m') + p v,  l = l * 2^(m - m') + sum p,
// and out = o / l.  Both products are register tiles fed from shared memory:
// a thread holds 8 queries x 4 keys of the scores (per four dims 12 vector
// reads for 128 FMAs, half the FMA rate's time) and 8 queries x 4 C values of
// the output.  Bound by the fp32 FMA rate: 2 (dk + dv) FLOP per pair.  K(j+1)
// is copied while the softmax and the second product of tile j run, V(j+1)
// under the next first product; one buffer each is enough for that.
#include "attention_common.cuh"
#include "launch_util.h"
#include "ptx.cuh"

namespace cb {

namespace {

constexpr int kBN = 64;

__device__ __forceinline__ void cp_async16(float* dst, const float* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// rows x width floats at dst (row pitch ld) from `valid` rows of `dim`
// elements `stride` apart; the rest is zero.  width is a multiple of 4.
template <typename T, bool VEC>
__device__ __forceinline__ void load_rows(float* dst, int ld, const T* src, long long stride, int rows, int valid,
                                          int dim, int width, int tid, int threads) {
  if constexpr (VEC && sizeof(T) == 4) {
    const int pieces = width >> 2;
    for (int e = tid; e < rows * pieces; e += threads) {
      const int r = e / pieces, d = (e - r * pieces) * 4;
      const bool ok = r < valid && d < dim;
      cp_async16(dst + r * ld + d, reinterpret_cast<const float*>(src) + (ok ? r * stride + d : 0), ok);
    }
  } else if constexpr (VEC) {
    const int pieces = (width + 7) >> 3;
    for (int e = tid; e < rows * pieces; e += threads) {
      const int r = e / pieces, d = (e - r * pieces) * 8;
      uint4 w = make_uint4(0, 0, 0, 0);
      if (r < valid && d < dim) w = *reinterpret_cast<const uint4*>(src + r * stride + d);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
      float f[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(u[i] << 16);
        f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
      }
      *reinterpret_cast<float4*>(dst + r * ld + d) = make_float4(f[0], f[1], f[2], f[3]);
      if (d + 4 < width) *reinterpret_cast<float4*>(dst + r * ld + d + 4) = make_float4(f[4], f[5], f[6], f[7]);
    }
  } else {
    for (int e = tid; e < rows * width; e += threads) {
      const int r = e / width, d = e - r * width;
      dst[r * ld + d] = r < valid && d < dim ? to_f32(src[r * stride + d]) : 0.f;
    }
  }
}

__host__ __device__ inline int qk_width(int dk) { return (dk + 3) & ~3; }
__host__ __device__ inline int qk_pitch(int dk) { return qk_width(dk) + 4; }

template <int BM, int C>
size_t simt_smem(int dk) {
  return sizeof(float) * (static_cast<size_t>(BM + kBN) * qk_pitch(dk) + kBN * 64 * C + kBN * (BM + 4)) + kBN * sizeof(int);
}

template <typename T, int BM, int C, bool VEC>
__global__ void __launch_bounds__(BM * 2, BM == 128 ? 1 : 2) attn_simt_kernel(AttnArgs a, int tiles) {
  constexpr int kThreads = BM * 2;
  extern __shared__ __align__(16) float smem[];
  const int ldk = qk_pitch(a.dk), wk = qk_width(a.dk);
  constexpr int ldv = 64 * C, ldp = BM + 4;
  float* Qs = smem;
  float* Ks = Qs + BM * ldk;
  float* Vs = Ks + kBN * ldk;
  float* Ps = Vs + kBN * ldv;
  int* doc_s = reinterpret_cast<int*>(Ps + kBN * ldp);
  __shared__ int s_next, s_dmin, s_dmax;

  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  // Last query tiles first: under a causal mask they are the longest.
  const int heads = a.B * a.Hq;
  const int tile = tiles - 1 - static_cast<int>(blockIdx.x / heads);
  const int bh = blockIdx.x % heads, b = bh / a.Hq, h = bh % a.Hq;
  const int i0 = tile * BM, rows = min(BM, a.Lq - i0);
  const T* q = static_cast<const T*>(a.q) + b * a.qs_b + static_cast<long long>(i0) * a.qs_l + h * a.qs_h;
  const T* k = static_cast<const T*>(a.k) + b * a.ks_b + (h / a.group) * a.ks_h;
  const T* v = static_cast<const T*>(a.v) + b * a.vs_b + (h / a.group) * a.vs_h;
  const SeqRule rule = seq_rule(a, b);
  const int hi_min = row_end(a, rule, i0), hi_max = row_end(a, rule, i0 + rows - 1);
  const int* doc_k = a.doc_k ? a.doc_k + static_cast<long long>(b) * a.Lk : nullptr;
  const float slope = a.slopes ? a.slopes[h] * kLog2e : 0.f;

  int hi[8], doc[8];
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const int i = i0 + ty * 8 + r;
    hi[r] = i < a.Lq ? row_end(a, rule, i) : 0;
    doc[r] = a.doc_q ? (i < a.Lq ? a.doc_q[static_cast<long long>(b) * a.Lq + i] : -1) : 0;
    if (doc[r] < 0) hi[r] = 0;
  }
  int dmin = 0, dmax = 0;
  if (a.doc_q) {
    if (tid == 0) s_dmin = 0x7fffffff, s_dmax = -1;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 8; ++r)
      if (doc[r] >= 0 && tx == 0) atomicMin(&s_dmin, doc[r]), atomicMax(&s_dmax, doc[r]);
    __syncthreads();
    dmin = s_dmin, dmax = s_dmax;
  }
  // First tile at or after j (a multiple of 64) with a key that may be visible.
  auto next = [&](int j) {
    if (!doc_k) return j;
    for (; j < hi_max; j += 4 * kThreads) {
      __syncthreads();
      if (tid == 0) s_next = 0x7fffffff;
      __syncthreads();
      for (int e = 0; e < 4; ++e) {
        const int key = j + tid + e * kThreads;
        if (key < hi_max) {
          const int d = doc_k[key];
          if (d >= dmin && d <= dmax) atomicMin(&s_next, key);
        }
      }
      __syncthreads();
      if (s_next != 0x7fffffff) return s_next & ~(kBN - 1);
    }
    return hi_max;
  };
  auto load_v = [&](int j) {
    load_rows<T, VEC>(Vs, ldv, v + j * a.vs_l, a.vs_l, kBN, min(kBN, rule.kv - j), a.dv, ldv, tid, kThreads);
    if (doc_k && tid < kBN) doc_s[tid] = j + tid < rule.kv ? doc_k[j + tid] : -1;
  };

  float m[8], l[8], acc[8][4 * C];
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    m[r] = kNegInf, l[r] = 0.f;
#pragma unroll
    for (int c = 0; c < 4 * C; ++c) acc[r][c] = 0.f;
  }

  int j0 = next(0);
  if (j0 < hi_max) {
    load_rows<T, VEC>(Qs, ldk, q, a.qs_l, BM, rows, a.dk, wk, tid, kThreads);
    load_rows<T, VEC>(Ks, ldk, k + j0 * a.ks_l, a.ks_l, kBN, min(kBN, rule.kv - j0), a.dk, wk, tid, kThreads);
    cp_async_commit();
    load_v(j0);
    cp_async_commit();
  }
  while (j0 < hi_max) {
    cp_async_wait<1>();
    __syncthreads();
    float s[8][4];
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c) s[r][c] = 0.f;
    const float* qr = Qs + ty * 8 * ldk;
    const float* kr = Ks + tx * ldk;
#pragma unroll 2
    for (int d = 0; d < wk; d += 4) {
      float4 kv[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) kv[c] = *reinterpret_cast<const float4*>(kr + 16 * c * ldk + d);
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const float4 qv = *reinterpret_cast<const float4*>(qr + r * ldk + d);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          s[r][c] = fmaf(qv.x, kv[c].x, s[r][c]);
          s[r][c] = fmaf(qv.y, kv[c].y, s[r][c]);
          s[r][c] = fmaf(qv.z, kv[c].z, s[r][c]);
          s[r][c] = fmaf(qv.w, kv[c].w, s[r][c]);
        }
      }
    }
    __syncthreads();
    const int jn = next(j0 + kBN);
    if (jn < hi_max)
      load_rows<T, VEC>(Ks, ldk, k + jn * a.ks_l, a.ks_l, kBN, min(kBN, rule.kv - jn), a.dk, wk, tid, kThreads);
    cp_async_commit();

    const bool masked = j0 + kBN > hi_min || doc_k;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const int at = i0 + ty * 8 + r + a.q_offset;
      float mx = kNegInf;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int j = j0 + tx + 16 * c;
        float x = score_log2(a, s[r][c], slope, abs(at - j));
        if (masked && !(j < hi[r] && (!doc_k || doc_s[tx + 16 * c] == doc[r]))) x = kNegInf;
        s[r][c] = x;
        mx = fmaxf(mx, x);
      }
#pragma unroll
      for (int o = 8; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, o));
      const float mn = fmaxf(m[r], mx), mu = mn == kNegInf ? 0.f : mn;
      const float corr = exp2_approx(m[r] - mu);
      m[r] = mn;
      l[r] *= corr;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        s[r][c] = exp2_approx(s[r][c] - mu);
        l[r] += s[r][c];
      }
#pragma unroll
      for (int c = 0; c < 4 * C; ++c) acc[r][c] *= corr;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float* p = Ps + (tx + 16 * c) * ldp + ty * 8;
      *reinterpret_cast<float4*>(p) = make_float4(s[0][c], s[1][c], s[2][c], s[3][c]);
      *reinterpret_cast<float4*>(p + 4) = make_float4(s[4][c], s[5][c], s[6][c], s[7][c]);
    }
    cp_async_wait<1>();
    __syncthreads();
#pragma unroll 2
    for (int key = 0; key < kBN; ++key) {
      const float4 p0 = *reinterpret_cast<const float4*>(Ps + key * ldp + ty * 8);
      const float4 p1 = *reinterpret_cast<const float4*>(Ps + key * ldp + ty * 8 + 4);
      const float p[8] = {p0.x, p0.y, p0.z, p0.w, p1.x, p1.y, p1.z, p1.w};
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const float4 vv = *reinterpret_cast<const float4*>(Vs + key * ldv + 64 * c + 4 * tx);
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          acc[r][4 * c] = fmaf(p[r], vv.x, acc[r][4 * c]);
          acc[r][4 * c + 1] = fmaf(p[r], vv.y, acc[r][4 * c + 1]);
          acc[r][4 * c + 2] = fmaf(p[r], vv.z, acc[r][4 * c + 2]);
          acc[r][4 * c + 3] = fmaf(p[r], vv.w, acc[r][4 * c + 3]);
        }
      }
    }
    __syncthreads();
    if (jn < hi_max) load_v(jn);
    cp_async_commit();
    j0 = jn;
  }
  cp_async_wait<0>();

  unsigned bad = 0;
#pragma unroll
  for (int r = 0; r < 8; ++r) {
#pragma unroll
    for (int o = 8; o; o >>= 1) l[r] += __shfl_xor_sync(~0u, l[r], o);
    const int i = i0 + ty * 8 + r;
    const float inv = l[r] == 0.f ? 0.f : 1.f / l[r];
    float probe = inv * 0.f;
#pragma unroll
    for (int c = 0; c < 4 * C; ++c) acc[r][c] *= inv, probe += acc[r][c] * 0.f;
    if (i < a.Lq) {
      if (!(probe == 0.f)) bad |= 1u << r;
      T* o = static_cast<T*>(a.o) + b * a.os_b + static_cast<long long>(i) * a.os_l + h * a.os_h;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int d = 64 * c + 4 * tx;
        if constexpr (VEC) {
          if (d < a.dv) {
            if constexpr (sizeof(T) == 4) {
              *reinterpret_cast<float4*>(o + d) = make_float4(acc[r][4 * c], acc[r][4 * c + 1], acc[r][4 * c + 2], acc[r][4 * c + 3]);
            } else {
              __nv_bfloat162 w[2] = {__floats2bfloat162_rn(acc[r][4 * c], acc[r][4 * c + 1]),
                                     __floats2bfloat162_rn(acc[r][4 * c + 2], acc[r][4 * c + 3])};
              *reinterpret_cast<uint2*>(o + d) = *reinterpret_cast<uint2*>(w);
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (d + e < a.dv) o[d + e] = from_f32<T>(acc[r][4 * c + e]);
        }
      }
    }
  }
  // Rows that met a non-finite value: again, key by key (attn_row).
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const unsigned who = __ballot_sync(~0u, (bad >> r) & 1);
    const int first = i0 + (tid >> 5) * 16 + r;
    __syncwarp();
    if (who & 0xffffu) attn_row<T>(a, b, h, first);
    if (who >> 16) attn_row<T>(a, b, h, first + 8);
  }
}

template <typename T, int BM, int C, bool VEC>
cudaError_t launch_one(const AttnArgs& a, cudaStream_t s) {
  const size_t smem = simt_smem<BM, C>(a.dk);
  const cudaError_t e = smem_attr_once<attn_simt_kernel<T, BM, C, VEC>>(smem);
  if (e != cudaSuccess) return e;
  const int tiles = (a.Lq + BM - 1) / BM;
  const long long ctas = static_cast<long long>(tiles) * a.B * a.Hq;
  if (ctas >= (1LL << 31)) return cudaErrorInvalidConfiguration;
  return launch_pdl(attn_simt_kernel<T, BM, C, VEC>, dim3(static_cast<unsigned>(ctas)), dim3(BM * 2), smem, s, a, tiles);
}

template <typename T, bool VEC>
cudaError_t launch_typed(const AttnArgs& a, int sms, cudaStream_t s) {
  // 128 queries per CTA feed the FMA units best; short or few sequences, which
  // would leave SMs without one, take 32.
  const bool small = static_cast<long long>(a.B) * a.Hq * ((a.Lq + 127) / 128) < sms;
  if (a.dv <= 64) return small ? launch_one<T, 32, 1, VEC>(a, s) : launch_one<T, 128, 1, VEC>(a, s);
  return small ? launch_one<T, 32, 2, VEC>(a, s) : launch_one<T, 128, 2, VEC>(a, s);
}

}  // namespace

cudaError_t launch_attn_simt(const AttnArgs& a, bool bf16, bool vec, int sms, cudaStream_t s) {
  if (bf16) return vec ? launch_typed<__nv_bfloat16, true>(a, sms, s) : launch_typed<__nv_bfloat16, false>(a, sms, s);
  return vec ? launch_typed<float, true>(a, sms, s) : launch_typed<float, false>(a, sms, s);
}

}  // namespace cb
