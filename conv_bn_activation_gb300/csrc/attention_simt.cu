// Attention in fp32 arithmetic on the CUDA cores: fp32 views, and bf16 views
// that the tensor-core kernel cannot address (attention_tc.cu).
//
// One CTA owns BM rows, (query, head) pairs that share a key head with the
// head running fastest, and walks the visible keys in tiles of 64 with the
// running maximum m and sum l of the softmax: for each tile
//   x = log2(e) * score, m' = max(m, max x), p = 2^(x - m'),
//   o = o * 2^(m - m') + p v,  l = l * 2^(m - m') + sum p,
// and out = o / l.  Both products are register tiles fed from shared memory:
// a thread holds 8 rows x 4 keys of the scores (per four dims 12 vector reads
// for 64 packed pairs of FMAs) and 8 rows x 2 C values of the output, C =
// ceil(dv / 32).  The FMA rate would bound it, 2 (dk + dv) FLOP per pair; the
// shared-memory reads do: 4096 tokens, 8 heads of 128 take 1.95 ms, 35 TFLOP/s
// or 0.47 of that rate, heads of 64 1.18 ms, 29 TFLOP/s.  K(j+1) is copied
// while the softmax and the second product of tile j run, V(j+1) under the
// next first product; one buffer each is enough for that.
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
// elements, row r at from(r); the rest is zero.  width is a multiple of 4; some: any readable address.
template <typename T, bool VEC, typename From>
__device__ __forceinline__ void load_rows(float* dst, int ld, From from, const T* some, int rows, int valid, int dim,
                                          int width, int tid, int threads) {
  if constexpr (VEC && sizeof(T) == 4) {
    const int pieces = width >> 2;
    for (int e = tid; e < rows * pieces; e += threads) {
      const int r = e / pieces, d = (e - r * pieces) * 4;
      const bool ok = r < valid && d < dim;
      cp_async16(dst + r * ld + d, reinterpret_cast<const float*>(ok ? from(r) + d : some), ok);
    }
  } else if constexpr (VEC) {
    const int pieces = (width + 7) >> 3;
    for (int e = tid; e < rows * pieces; e += threads) {
      const int r = e / pieces, d = (e - r * pieces) * 8;
      uint4 w = make_uint4(0, 0, 0, 0);
      if (r < valid && d < dim) w = *reinterpret_cast<const uint4*>(from(r) + d);
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
      dst[r * ld + d] = r < valid && d < dim ? to_f32(from(r)[d]) : 0.f;
    }
  }
}

__host__ __device__ inline int qk_width(int dk) { return (dk + 3) & ~3; }
__host__ __device__ inline int qk_pitch(int dk) { return qk_width(dk) + 4; }

template <int BM, int C>
size_t simt_smem(int dk) {
  return sizeof(float) * (static_cast<size_t>(BM + kBN) * qk_pitch(dk) + kBN * 32 * C + kBN * (BM + 4)) + kBN * sizeof(int);
}

template <typename T, int BM, int C, bool VEC>
__global__ void __launch_bounds__(BM * 2, BM == 128 ? 1 : 2) attn_simt_kernel(AttnArgs a, int tiles) {
  constexpr int kThreads = BM * 2;
  extern __shared__ __align__(16) float smem[];
  const int ldk = qk_pitch(a.dk), wk = qk_width(a.dk);
  constexpr int ldv = 32 * C, ldp = BM + 4;
  float* Qs = smem;
  float* Ks = Qs + BM * ldk;
  float* Vs = Ks + kBN * ldk;
  float* Ps = Vs + kBN * ldv;
  int* doc_s = reinterpret_cast<int*>(Ps + kBN * ldp);
  __shared__ int s_next, s_dmin, s_dmax;

  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  // Last rows first: under a causal mask they see the most keys.
  const int hkv = a.Hq / a.group, seqs = a.B * hkv;
  const int tile = tiles - 1 - static_cast<int>(blockIdx.x / seqs);
  const int bh = blockIdx.x % seqs, b = bh / hkv, hk = bh % hkv;
  const int r0 = tile * BM, rows = min(BM, a.Lq * a.group - r0);  // row r: query r / group, head r % group of the key head's
  const T* q = static_cast<const T*>(a.q) + b * a.qs_b + hk * a.group * a.qs_h;
  const T* k = static_cast<const T*>(a.k) + b * a.ks_b + hk * a.ks_h;
  const T* v = static_cast<const T*>(a.v) + b * a.vs_b + hk * a.vs_h;
  const SeqRule rule = seq_rule(a, b);
  const int hi_min = row_end(a, rule, r0 / a.group), hi_max = row_end(a, rule, (r0 + rows - 1) / a.group);
  const int* doc_k = a.doc_k ? a.doc_k + static_cast<long long>(b) * a.Lk : nullptr;
  const float inv_cap = a.softcap > 0.f ? a.scale / a.softcap : 0.f, cap_log2 = a.softcap * kLog2e, c_scale = a.scale * kLog2e;

  int at[8], hi[8], doc[8];  // at: a row's place among the keys
  float slope[8];
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const int row = r0 + ty * 8 + r, i = row / a.group;
    const bool real = ty * 8 + r < rows;
    at[r] = i + a.q_offset;
    hi[r] = real ? row_end(a, rule, i) : 0;
    doc[r] = a.doc_q ? (real ? a.doc_q[static_cast<long long>(b) * a.Lq + i] : -1) : 0;
    if (doc[r] < 0) hi[r] = 0;
    slope[r] = a.slopes ? a.slopes[hk * a.group + row % a.group] * kLog2e : 0.f;
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
    load_rows<T, VEC>(Vs, ldv, [&](int r) { return v + (j + r) * a.vs_l; }, v, kBN, min(kBN, rule.kv - j), a.dv, ldv, tid, kThreads);
    if (doc_k && tid < kBN) doc_s[tid] = j + tid < rule.kv ? doc_k[j + tid] : -1;
  };

  float m[8], l[8];
  f2 acc[4][2 * C];  // rows 2 r and 2 r + 1
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    m[r] = kNegInf, l[r] = 0.f;
#pragma unroll
    for (int c = 0; c < 2 * C; ++c) acc[r >> 1][c] = 0;
  }

  int j0 = next(0);
  if (j0 < hi_max) {
    load_rows<T, VEC>(Qs, ldk, [&](int r) { return q + (r0 + r) / a.group * a.qs_l + (r0 + r) % a.group * a.qs_h; }, q, BM, rows, a.dk, wk, tid, kThreads);
    load_rows<T, VEC>(Ks, ldk, [&](int r) { return k + (j0 + r) * a.ks_l; }, k, kBN, min(kBN, rule.kv - j0), a.dk, wk, tid, kThreads);
    cp_async_commit();
    load_v(j0);
    cp_async_commit();
  }
  while (j0 < hi_max) {
    cp_async_wait<1>();
    __syncthreads();
    // Products of even and of odd dims apart: two FMAs per instruction, operands as they lie.
    f2 s2[8][4];
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c) s2[r][c] = 0;
    const float* qr = Qs + ty * 8 * ldk;
    const float* kr = Ks + tx * ldk;
#pragma unroll 2
    for (int d = 0; d < wk; d += 4) {
      ulonglong2 kv[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) kv[c] = *reinterpret_cast<const ulonglong2*>(kr + 16 * c * ldk + d);
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const ulonglong2 qv = *reinterpret_cast<const ulonglong2*>(qr + r * ldk + d);
#pragma unroll
        for (int c = 0; c < 4; ++c) s2[r][c] = fma2(qv.y, kv[c].y, fma2(qv.x, kv[c].x, s2[r][c]));
      }
    }
    float s[8][4];
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float even, odd;
        unpack2(s2[r][c], even, odd);
        s[r][c] = even + odd;
      }
    __syncthreads();
    const int jn = next(j0 + kBN);
    if (jn < hi_max)
      load_rows<T, VEC>(Ks, ldk, [&](int r) { return k + (jn + r) * a.ks_l; }, k, kBN, min(kBN, rule.kv - jn), a.dk, wk, tid, kThreads);
    cp_async_commit();

    const bool masked = j0 + kBN > hi_min || doc_k;
    float corr[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      float mx = kNegInf;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int j = j0 + tx + 16 * c;
        float x = a.softcap > 0.f ? cap_log2 * tanhf(s[r][c] * inv_cap) : s[r][c] * c_scale;
        if (a.slopes) x = fmaf(-slope[r], static_cast<float>(abs(at[r] - j)), x);
        if (masked && !(j < hi[r] && (!doc_k || doc_s[tx + 16 * c] == doc[r]))) x = kNegInf;
        s[r][c] = x;
        mx = fmaxf(mx, x);
      }
#pragma unroll
      for (int o = 8; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, o));
      const float mn = fmaxf(m[r], mx), mu = mn == kNegInf ? 0.f : mn;
      corr[r] = exp2_approx(m[r] - mu);
      m[r] = mn;
      l[r] *= corr[r];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        s[r][c] = exp2_approx(s[r][c] - mu);
        l[r] += s[r][c];
      }
      if (r & 1) {
        const f2 f = pack2(corr[r - 1], corr[r]);
#pragma unroll
        for (int c = 0; c < 2 * C; ++c) acc[r >> 1][c] = mul2(acc[r >> 1][c], f);
      }
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
      const ulonglong2 p0 = *reinterpret_cast<const ulonglong2*>(Ps + key * ldp + ty * 8);
      const ulonglong2 p1 = *reinterpret_cast<const ulonglong2*>(Ps + key * ldp + ty * 8 + 4);
      const f2 p[4] = {p0.x, p0.y, p1.x, p1.y};
      float vv[2 * C];
#pragma unroll
      for (int c = 0; c + 2 <= C; c += 2) {
        const float4 w = *reinterpret_cast<const float4*>(Vs + key * ldv + 32 * c + 4 * tx);
        vv[2 * c] = w.x, vv[2 * c + 1] = w.y, vv[2 * c + 2] = w.z, vv[2 * c + 3] = w.w;
      }
      if constexpr (C & 1) {
        const float2 w = *reinterpret_cast<const float2*>(Vs + key * ldv + 32 * (C - 1) + 2 * tx);
        vv[2 * C - 2] = w.x, vv[2 * C - 1] = w.y;
      }
#pragma unroll
      for (int c = 0; c < 2 * C; ++c) {
        const f2 v2 = pack2(vv[c], vv[c]);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[r][c] = fma2(p[r], v2, acc[r][c]);
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
    const int row = r0 + ty * 8 + r;
    const float inv = l[r] == 0.f ? 0.f : 1.f / l[r];
    float probe = inv * 0.f;
    float y[2 * C];
#pragma unroll
    for (int c = 0; c < 2 * C; ++c) {
      float lo, up;
      unpack2(acc[r >> 1][c], lo, up);
      y[c] = (r & 1 ? up : lo) * inv;
      probe += y[c] * 0.f;
    }
    if (ty * 8 + r < rows) {
      if (!(probe == 0.f)) bad |= 1u << r;
      T* o = static_cast<T*>(a.o) + b * a.os_b + row / a.group * a.os_l + (hk * a.group + row % a.group) * a.os_h;
#pragma unroll
      for (int c = 0; c < C; ++c) {  // two values at a time; their dims as the products took them
        const int d = (C & 1) && c == C - 1 ? 32 * c + 2 * tx : 32 * (c & ~1) + 4 * tx + 2 * (c & 1);
        if constexpr (VEC) {
          if (d < a.dv) {
            if constexpr (sizeof(T) == 4) *reinterpret_cast<float2*>(o + d) = make_float2(y[2 * c], y[2 * c + 1]);
            else *reinterpret_cast<__nv_bfloat162*>(o + d) = __floats2bfloat162_rn(y[2 * c], y[2 * c + 1]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (d + e < a.dv) o[d + e] = from_f32<T>(y[2 * c + e]);
        }
      }
    }
  }
  // Rows that met a hidden value that is not finite: again, key by key. This warp's 16 rows, one per lane.
  const int lane = tid & 31, row = r0 + (tid >> 5) * 16 + lane;
  unsigned odd = 0;
  float sum = 0.f;
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const unsigned who = __ballot_sync(~0u, (bad >> r) & 1);
    odd |= (who & 0xffffu ? 1u << r : 0u) | (who >> 16 ? 256u << r : 0u);
    const float x = __shfl_sync(~0u, l[r], lane & 8 ? 16 : 0);
    if ((lane & 7) == r) sum = x;
  }
  if (odd) {
    const bool mine = lane < 16 && (odd >> lane) & 1;
    const int i = mine ? row / a.group : 0, my_doc = mine && a.doc_q ? a.doc_q[static_cast<long long>(b) * a.Lq + i] : 0;
    const int end = min(rule.kv, (hi_max + kBN - 1) / kBN * kBN);
    unsigned again = rows_to_redo<T, VEC>(a, b, hk, end, mine, mine && my_doc >= 0 ? row_end(a, rule, i) : 0, my_doc, sum);
    for (; again; again &= again - 1) {
      const int r = row - lane + __ffs(again) - 1;
      attn_row<T, VEC>(a, b, hk * a.group + r % a.group, r / a.group);
    }
  }
}

template <typename T, int BM, int C, bool VEC>
cudaError_t launch_one(const AttnArgs& a, cudaStream_t s) {
  const size_t smem = simt_smem<BM, C>(a.dk);
  const cudaError_t e = smem_attr_once<attn_simt_kernel<T, BM, C, VEC>>(smem);
  if (e != cudaSuccess) return e;
  const int tiles = static_cast<int>((static_cast<long long>(a.Lq) * a.group + BM - 1) / BM);
  const long long ctas = static_cast<long long>(tiles) * a.B * (a.Hq / a.group);
  if (ctas >= (1LL << 31)) return cudaErrorInvalidConfiguration;
  return launch_pdl(attn_simt_kernel<T, BM, C, VEC>, dim3(static_cast<unsigned>(ctas)), dim3(BM * 2), smem, s, a, tiles);
}

template <typename T, bool VEC, int BM>
cudaError_t launch_rows(const AttnArgs& a, cudaStream_t s) {
  if (a.dv <= 64) return launch_one<T, BM, 2, VEC>(a, s);
  return a.dv <= 96 ? launch_one<T, BM, 3, VEC>(a, s) : launch_one<T, BM, 4, VEC>(a, s);
}

// 64 rows per CTA, two CTAs per SM, or 128 where two of 64 do not fit its shared
// memory (128 dims: 1.95 ms for 4096 tokens and 8 heads against 2.69); 32 rows
// where the larger tile, empty rows and a last partial wave counted, takes
// longer.  A full SM works through 32 rows a quarter (128 dims: a half) slower,
// and tiles alone on theirs take as long as 64 (4096 tokens, 8 heads of 64: 1.18
// ms with 64, 1.25 with 32; 58 sequences of 76 tokens, 4 heads on 2: 44 and 28 us).
template <typename T, bool VEC>
cudaError_t launch_typed(const AttnArgs& a, int sms, cudaStream_t s) {
  const long long rows = static_cast<long long>(a.Lq) * a.group, seqs = static_cast<long long>(a.B) * (a.Hq / a.group);
  const bool two = 2 * ((a.dv <= 64 ? simt_smem<64, 2>(a.dk) : a.dv <= 96 ? simt_smem<64, 3>(a.dk) : simt_smem<64, 4>(a.dk)) + 1280) <= 233472;
  auto cost = [&](int bm) {
    const long long c = ((rows + bm - 1) / bm * seqs + sms - 1) / sms * bm;
    return c > 64 ? c : 64;
  };
  if (two) return 5 * cost(32) < 4 * cost(64) ? launch_rows<T, VEC, 32>(a, s) : launch_rows<T, VEC, 64>(a, s);
  return 3 * cost(32) < 2 * cost(128) ? launch_rows<T, VEC, 32>(a, s) : launch_rows<T, VEC, 128>(a, s);
}

}  // namespace

cudaError_t launch_attn_simt(const AttnArgs& a, bool bf16, bool vec, int sms, cudaStream_t s) {
  if (bf16) return vec ? launch_typed<__nv_bfloat16, true>(a, sms, s) : launch_typed<__nv_bfloat16, false>(a, sms, s);
  return vec ? launch_typed<float, true>(a, sms, s) : launch_typed<float, false>(a, sms, s);
}

}  // namespace cb
