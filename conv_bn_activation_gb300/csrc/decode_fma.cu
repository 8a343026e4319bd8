// The decode kernel's arithmetic for fp32 caches (decode_stream.cuh): FMAs, so
// that products and sums keep fp32 precision.  A warp's step is 8 keys.  For
// the scores four lanes share a key, each a quarter of its dims; for the output
// each lane holds DV / 32 of the values' dims and every head.  NH heads per
// item: 4 NH FLOP per element of the cache against the FMA pipe's 21 per byte
// at the memory's rate.
#include "decode_stream.cuh"

namespace cb {

namespace {

__device__ __forceinline__ float4 lds4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

template <int DK_, int DV_, int NH, bool ROWS>
struct FmaPolicy {
  using T = float;
  static constexpr int DK = DK_, DV = DV_, kStep = 8, kStages = 3, kHeads = NH;
  static constexpr bool kRows = ROWS;
  static constexpr int kQBytes = NH * DK * 4;                          // q, one copy per CTA
  static constexpr int kPStride = NH < 4 ? 4 : NH;                     // weights [8 keys][heads] per warp
  static constexpr int kExtra = kQBytes + kDecodeWarps * 8 * kPStride * 4;
  static constexpr int kKeyBytes = DK * 4, kValBytes = DV * 4;
  static constexpr int OWN = (NH + 3) / 4;                             // heads whose softmax a lane does
  static constexpr int EV = DV / 32;                                   // values' dims per lane
  // Eight lanes of a shared-memory access hold two keys' four pieces: keys of
  // odd number take the other half of 128 bytes.
  static __device__ __forceinline__ constexpr int swizzle(int row) { return ((row & 1) << 2) | ((row & 6) >> 1); }

  DecodeScore score;
  int key, sub, lane, heads;
  uint32_t q_addr, p_addr;
  float* p_mine;
  RowRule rule[OWN];
  float slope[OWN], m[OWN], l[OWN], o[NH][EV];

  __device__ __forceinline__ FmaPolicy(const DecodeArgs& a, const AttnArgs& rw, const Piece& pc, uint8_t* after) : score(a) {
    lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    key = lane >> 2, sub = lane & 3, heads = pc.heads;
    float* q = reinterpret_cast<float*>(after);
    for (int e = threadIdx.x; e < NH * DK; e += kDecodeThreads) {
      const int h = e / DK, d = e % DK;
      q[e] = h < heads && d < a.dk ? query_row<ROWS, float>(a, rw, pc, h)[d] : 0.f;
    }
    __syncthreads();
    q_addr = smem_u32(q);
    p_mine = reinterpret_cast<float*>(after + kQBytes) + warp * 8 * kPStride;
    p_addr = smem_u32(p_mine);
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
      const int h = sub + 4 * i;
      slope[i] = slope_of(a, rw, pc, h, ROWS);
      if constexpr (ROWS) rule[i] = row_rule(a, rw, pc, h);
      m[i] = kNegInf;
      l[i] = 0.f;
    }
#pragma unroll
    for (int h = 0; h < NH; ++h)
#pragma unroll
      for (int e = 0; e < EV; ++e) o[h][e] = 0.f;
  }

  template <bool>
  __device__ __forceinline__ void step(uint32_t ks, uint32_t vs, unsigned lv, int far, int doc) {
    float dot[NH];
#pragma unroll
    for (int h = 0; h < NH; ++h) dot[h] = 0.f;
    const uint32_t row = ks + key * kKeyBytes, sw = swizzle(key);
#pragma unroll
    for (int p = 0; p < DK / 16; ++p) {
      const float4 k = lds4(row + (((4 * p + sub) ^ sw) * 16));
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        const float4 q = lds4(q_addr + (h * DK + (4 * p + sub) * 4) * 4);
        dot[h] = fmaf(q.x, k.x, fmaf(q.y, k.y, fmaf(q.z, k.z, fmaf(q.w, k.w, dot[h]))));
      }
    }
    // This lane's heads sub, sub + 4, ... of its key.
    const bool exists = (lv >> key) & 1;
    const int my_doc = ROWS ? __shfl_sync(~0u, doc, key) : 0;
    float x[OWN], own[1][OWN];
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
      // The four lanes' sums of four heads, each lane left with its own head's.
      const float d0 = dot[4 * i], d1 = 4 * i + 1 < NH ? dot[(4 * i + 1) % NH] : 0.f;
      const float d2 = 4 * i + 2 < NH ? dot[(4 * i + 2) % NH] : 0.f, d3 = 4 * i + 3 < NH ? dot[(4 * i + 3) % NH] : 0.f;
      const bool hi = sub & 2, odd = sub & 1;
      const float e0 = (hi ? d2 : d0) + __shfl_xor_sync(~0u, hi ? d0 : d2, 2);
      const float e1 = (hi ? d3 : d1) + __shfl_xor_sync(~0u, hi ? d1 : d3, 2);
      own[0][i] = (odd ? e1 : e0) + __shfl_xor_sync(~0u, odd ? e0 : e1, 1);
    }
    score(own);
    bool grow = false;
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
      if constexpr (ROWS) {
        const int j = far + key;
        const bool seen = exists && j < rule[i].hi && my_doc == rule[i].doc;
        x[i] = seen ? fmaf(-slope[i], static_cast<float>(abs(rule[i].at - j)), own[0][i]) : kNegInf;
      } else {
        x[i] = exists ? fmaf(-slope[i], static_cast<float>(far - key), own[0][i]) : kNegInf;
      }
      grow |= x[i] > m[i] + kDecodeGrowth;
    }
    if (__any_sync(~0u, grow)) {  // only then are the maxima taken
      float f[OWN];
#pragma unroll
      for (int i = 0; i < OWN; ++i) {
        float y = x[i];
        y = fmaxf(y, __shfl_xor_sync(~0u, y, 4));
        y = fmaxf(y, __shfl_xor_sync(~0u, y, 8));
        y = fmaxf(y, __shfl_xor_sync(~0u, y, 16));
        const float mn = fmaxf(m[i], y);
        f[i] = mn == kNegInf ? 1.f : exp2_approx(m[i] - mn);
        m[i] = mn;
        l[i] *= f[i];
      }
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        const float fh = __shfl_sync(~0u, f[h / 4], h % 4);
#pragma unroll
        for (int e = 0; e < EV; ++e) o[h][e] *= fh;
      }
    }
    __syncwarp();  // the last step's weights were read
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
      const float p = exp2_approx(x[i] - (m[i] == kNegInf ? 0.f : m[i]));
      l[i] += p;
      p_mine[key * kPStride + sub + 4 * i] = p;
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float v[EV];
      const uint32_t at = vs + k * kValBytes;
      if constexpr (EV == 4) {
        const float4 w = lds4(at + ((lane ^ swizzle(k)) * 16));
        v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
      } else {
        asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];"
                     : "=f"(v[0]), "=f"(v[1])
                     : "r"(at + (((lane >> 1) ^ swizzle(k)) * 16) + (lane & 1) * 8)
                     : "memory");
      }
#pragma unroll
      for (int h4 = 0; h4 < NH; h4 += 4) {
        const float4 w = lds4(p_addr + (k * kPStride + h4) * 4);
        const float p[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int h = 0; h < 4; ++h)
          if (h4 + h < NH)
#pragma unroll
            for (int e = 0; e < EV; ++e) o[h4 + h][e] = fmaf(p[h], v[e], o[h4 + h][e]);
      }
    }
  }

  __device__ __forceinline__ void store(float* res, float* ms, float* ls) {
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
      float y = l[i];
      y += __shfl_xor_sync(~0u, y, 4);
      y += __shfl_xor_sync(~0u, y, 8);
      y += __shfl_xor_sync(~0u, y, 16);
      if (key == 0 && sub + 4 * i < NH) ms[sub + 4 * i] = m[i], ls[sub + 4 * i] = y;
    }
#pragma unroll
    for (int h = 0; h < NH; ++h)
      if (h < heads)
#pragma unroll
        for (int e = 0; e < EV; ++e) res[h * DV + lane * EV + e] = o[h][e];
  }
};

template <int DK, int DV>
cudaError_t launch_dims(const DecodeArgs& a, cudaStream_t s) {
  if (a.item_heads <= 1) return launch_decode_stream<FmaPolicy<DK, DV, 1, false>>(a, s);
  if (a.item_heads <= 2) return launch_decode_stream<FmaPolicy<DK, DV, 2, false>>(a, s);
  if (a.item_heads <= 4) return launch_decode_stream<FmaPolicy<DK, DV, 4, false>>(a, s);
  return launch_decode_stream<FmaPolicy<DK, DV, 8, false>>(a, s);
}

}  // namespace

cudaError_t launch_decode_fma(const DecodeArgs& a, cudaStream_t s) {
  if (a.dk <= 64) return a.dv <= 64 ? launch_dims<64, 64>(a, s) : launch_dims<64, 128>(a, s);
  return a.dv <= 64 ? launch_dims<128, 64>(a, s) : launch_dims<128, 128>(a, s);
}

cudaError_t launch_rows_fma(const DecodeArgs& a, const AttnArgs& rw, cudaStream_t s) {
  const long long ctas = static_cast<long long>(a.B) * a.Hkv * a.chunks * a.split;
  if (a.dk <= 64)
    return a.dv <= 64 ? launch_whole<FmaPolicy<64, 64, 8, true>>(a, rw, ctas, s) : launch_whole<FmaPolicy<64, 128, 8, true>>(a, rw, ctas, s);
  return a.dv <= 64 ? launch_whole<FmaPolicy<128, 64, 8, true>>(a, rw, ctas, s) : launch_whole<FmaPolicy<128, 128, 8, true>>(a, rw, ctas, s);
}

}  // namespace cb
