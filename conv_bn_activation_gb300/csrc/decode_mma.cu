// The decode kernel's arithmetic for bf16 caches (decode_stream.cuh): warp-level
// MMAs.  With 8 query heads to a key head the products are 8 FLOP per byte, too
// much conversion and FMA work for the CUDA cores at the memory's rate (a bf16
// value feeds 8 FMAs after one conversion; measured 5.6x slower), and too
// little for tcgen05, whose 128 rows would hold 8 queries and whose operands
// would cross shared memory no faster.  Keys (then the values' dims) are the
// MMAs' 16 rows, 8 heads their columns, NB of them per item:
//   S^T[16 keys x 8 heads] = K Q^T,  P = 2^(x - m),  O^T[dv x 8 heads] += V^T P^T.
// l sums the weights as rounded to bf16 for the second product, so their
// rounding largely cancels.  Eight sequences of up to 131072 tokens, 8 key
// heads of 128: 480 us, 6.7 TB/s (the measured copy rate).
#include "decode_stream.cuh"

namespace cb {

namespace {

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// The transpose of an 8 x 8 matrix of 16-bit elements held as an MMA fragment.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
// d (16 x 8, fp32) += a (16 x 16, bf16) * b (16 x 8, bf16)
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int DK_, int DV_, int NB, bool ROWS>
struct MmaPolicy {
  using T = __nv_bfloat16;
  static constexpr int DK = DK_, DV = DV_, kStep = 16, kStages = 3, kHeads = 8 * NB, kExtra = 0;
  static constexpr bool kRows = ROWS;
  static constexpr int kKeyBytes = DK * 2, kValBytes = DV * 2;
  static __device__ __forceinline__ constexpr int swizzle(int row) { return row & 7; }

  DecodeScore score;
  bool bias;
  int g, t4, heads;
  uint32_t k_src, v_src;  // this lane's ldmatrix rows
  // Q^T as the MMA's B operand: head g of each 8, elements 2 t4 and 2 t4 + 8 of each 16.
  uint32_t qf[DK / 16][NB][2];
  // This thread's heads are 8 nb + 2 t4 and the one after.
  RowRule rule[NB][2];
  float slope[NB][2], m[NB][2], l[NB][2], o[DV / 16][NB][4];

  __device__ __forceinline__ MmaPolicy(const DecodeArgs& a, const AttnArgs& rw, const Piece& pc, uint8_t*) : score(a) {
    const int lane = threadIdx.x & 31;
    g = lane >> 2, t4 = lane & 3, heads = pc.heads;
    bias = ROWS ? rw.slopes != nullptr : a.slopes != nullptr;
    k_src = ((lane & 7) + 8 * ((lane >> 3) & 1)) * kKeyBytes + (((lane >> 4) ^ (lane & 7)) * 16);
    v_src = ((lane & 7) + 8 * (lane >> 4)) * kValBytes + ((((lane >> 3) & 1) ^ (lane & 7)) * 16);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int hd = g + 8 * nb;
      const T* q = query_row<ROWS, T>(a, rw, pc, hd < heads ? hd : 0);
#pragma unroll
      for (int s = 0; s < DK / 16; ++s)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int d = 16 * s + 2 * t4 + 8 * r;
          uint32_t w = 0;
          if (hd < heads && d < a.dk)  // dk is even; rows are 16-byte aligned, a decode query need not be
            w = ROWS ? *reinterpret_cast<const uint32_t*>(q + d)
                     : static_cast<uint32_t>(__bfloat16_as_ushort(q[d])) | (static_cast<uint32_t>(__bfloat16_as_ushort(q[d + 1])) << 16);
          qf[s][nb][r] = w;
        }
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int hd = 8 * nb + 2 * t4 + e;
        slope[nb][e] = slope_of(a, rw, pc, hd, ROWS);
        if constexpr (ROWS) rule[nb][e] = row_rule(a, rw, pc, hd);
        m[nb][e] = kNegInf;
        l[nb][e] = 0.f;
      }
#pragma unroll
      for (int d = 0; d < DV / 16; ++d)
#pragma unroll
        for (int r = 0; r < 4; ++r) o[d][nb][r] = 0.f;
    }
  }

  // 16 keys at ks / vs; bit x of lv: key x exists; far: the first key's distance
  // from the query (ROWS: its place); doc: the document of key lane % 16 (ROWS).
  // EAGER: the maxima are taken only when a score passes the last ones by kDecodeGrowth.
  template <bool EAGER>
  __device__ __forceinline__ void step(uint32_t ks, uint32_t vs, unsigned lv, int far, int doc) {
    float s[NB][4];  // element r: key g + 8 (r >> 1), head 8 nb + 2 t4 + (r & 1)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int r = 0; r < 4; ++r) s[nb][r] = 0.f;
#pragma unroll
    for (int d = 0; d < DK / 16; ++d) {
      uint32_t f[4];
      ldsm4((ks + k_src + (d >> 2) * 128) ^ ((d & 3) * 32), f);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) mma16816(s[nb], f, qf[d][nb][0], qf[d][nb][1]);
    }
    score(s);  // x = log2(e) * score
    const float dist = static_cast<float>(far - g);
    const int doc0 = ROWS ? __shfl_sync(~0u, doc, g) : 0, doc1 = ROWS ? __shfl_sync(~0u, doc, g + 8) : 0;
    bool grow = false;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float x = s[nb][r];
        if constexpr (ROWS) {
          const RowRule& w = rule[nb][r & 1];
          const int j = far + g + 8 * (r >> 1);
          if (bias) x = fmaf(-slope[nb][r & 1], static_cast<float>(abs(w.at - j)), x);
          if (j >= w.hi || (r < 2 ? doc0 : doc1) != w.doc) x = kNegInf;
        } else {
          if (bias) x = fmaf(-slope[nb][r & 1], dist - 8.f * (r >> 1), x);
        }
        if (lv != 0xffffu && !((lv >> (g + 8 * (r >> 1))) & 1)) x = kNegInf;
        s[nb][r] = x;
        if (EAGER) grow |= x > m[nb][r & 1] + kDecodeGrowth;
      }
    }
    float mx[NB][2];
    auto maxima = [&] {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float y = fmaxf(s[nb][e], s[nb][2 + e]);
          y = fmaxf(y, __shfl_xor_sync(~0u, y, 4));
          y = fmaxf(y, __shfl_xor_sync(~0u, y, 8));
          y = fmaxf(y, __shfl_xor_sync(~0u, y, 16));
          mx[nb][e] = y;
          if (!EAGER) grow |= y > m[nb][e] + kDecodeGrowth;
        }
    };
    if (!EAGER) maxima();
    if (__any_sync(~0u, grow)) {
      if (EAGER) maxima();
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float mn = fmaxf(m[nb][e], mx[nb][e]);
          const float f = mn == kNegInf ? 1.f : exp2_approx(m[nb][e] - mn);
          m[nb][e] = mn;
          l[nb][e] *= f;
#pragma unroll
          for (int d = 0; d < DV / 16; ++d) o[d][nb][e] *= f, o[d][nb][2 + e] *= f;
        }
    }
    uint32_t p[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const float mu0 = m[nb][0] == kNegInf ? 0.f : m[nb][0], mu1 = m[nb][1] == kNegInf ? 0.f : m[nb][1];
#pragma unroll
      for (int r = 0; r < 2; ++r) {  // keys 8 r .. + 8
        const __nv_bfloat162 w = __floats2bfloat162_rn(exp2_approx(s[nb][2 * r] - mu0), exp2_approx(s[nb][2 * r + 1] - mu1));
        l[nb][0] += __low2float(w);
        l[nb][1] += __high2float(w);
        p[nb][r] = transpose8(*reinterpret_cast<const uint32_t*>(&w));
      }
    }
#pragma unroll
    for (int d = 0; d < DV / 16; ++d) {  // values 16 d .. + 16 of the 16 keys
      uint32_t f[4];
      ldsm4_t((vs + v_src + (d >> 2) * 128) ^ ((d & 3) * 32), f);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) mma16816(o[d][nb], f, p[nb][0], p[nb][1]);
    }
  }

  // This warp's results: res[heads][DV] unnormalised, its maxima and sums.
  __device__ __forceinline__ void store(float* res, float* ms, float* ls) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float y = l[nb][e];
        y += __shfl_xor_sync(~0u, y, 4);
        y += __shfl_xor_sync(~0u, y, 8);
        y += __shfl_xor_sync(~0u, y, 16);
        const int hd = 8 * nb + 2 * t4 + e;
        if (g == 0) ms[hd] = m[nb][e], ls[hd] = y;
        if (hd < heads)
#pragma unroll
          for (int d = 0; d < DV / 16; ++d) {
            res[hd * DV + 16 * d + g] = o[d][nb][e];
            res[hd * DV + 16 * d + g + 8] = o[d][nb][2 + e];
          }
      }
  }
};

template <int DK, int DV>
cudaError_t launch_dims(const DecodeArgs& a, cudaStream_t s) {
  return a.item_heads <= 8 ? launch_decode_stream<MmaPolicy<DK, DV, 1, false>>(a, s)
                           : launch_decode_stream<MmaPolicy<DK, DV, 2, false>>(a, s);
}

}  // namespace

cudaError_t launch_decode_mma(const DecodeArgs& a, cudaStream_t s) {
  if (a.dk <= 64) return a.dv <= 64 ? launch_dims<64, 64>(a, s) : launch_dims<64, 128>(a, s);
  return a.dv <= 64 ? launch_dims<128, 64>(a, s) : launch_dims<128, 128>(a, s);
}

cudaError_t launch_rows_mma(const DecodeArgs& a, const AttnArgs& rw, cudaStream_t s) {
  const long long ctas = static_cast<long long>(a.B) * a.Hkv * a.chunks * a.split;
  if (a.dk <= 64)
    return a.dv <= 64 ? launch_whole<MmaPolicy<64, 64, 2, true>>(a, rw, ctas, s) : launch_whole<MmaPolicy<64, 128, 2, true>>(a, rw, ctas, s);
  return a.dv <= 64 ? launch_whole<MmaPolicy<128, 64, 2, true>>(a, rw, ctas, s) : launch_whole<MmaPolicy<128, 128, 2, true>>(a, rw, ctas, s);
}

}  // namespace cb
