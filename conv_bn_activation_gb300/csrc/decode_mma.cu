// Attention of one new token per sequence over a paged bf16 cache whose rows
// are whole 16-byte pieces (cb_attention_decode; decode_common.cuh says how
// tokens are dealt to the CTAs).
//
// Bound by HBM: 2 (dk + dv) bytes per cached token and key head, read once.
// The query heads that share a key head ride along: with 8 of them the
// products are 8 FLOP per byte, too much conversion and FMA work for the CUDA
// cores at the memory's rate (a bf16 value feeds 8 FMAs after one conversion;
// measured 5.6x slower), and too little for tcgen05, whose 128 rows would hold
// 8 queries and whose operands would cross shared memory no faster. So the
// products are warp-level MMAs with the keys (then the values' dims) as their
// 16 rows and 8 heads as their columns, NB of them per item:
//   S^T[16 keys x 8 heads] = K Q^T,  P = 2^(x - m),  O^T[dv x 8 heads] += V^T P^T.
// Each warp walks its own 16 keys of every 64-token tile with its own ring of
// cp.async copies and its own maximum, sum and O, so nothing synchronises
// inside a run; the four warps are joined when an item's piece ends. O is
// rescaled only when a maximum grows by more than 2^8. l sums the weights as
// rounded to bf16 for the second product, so their rounding largely cancels.
#include "decode_common.cuh"
#include "launch_util.h"
#include "ptx.cuh"

namespace cb {

namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kStep = 16;      // keys per warp and step
constexpr int kStages = 3;
constexpr float kGrowth = 8.f;
static_assert(kWarps * kStep == kDecodeTile, "a tile is one step of every warp");

template <int DK, int DV>
constexpr int stage_bytes() { return kStep * (DK + DV) * 2; }
template <int DK, int DV>
constexpr int ring_bytes() {  // also holds the warps' results when a piece ends
  return kWarps * kStages * stage_bytes<DK, DV>();
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
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

template <int DK, int DV, int NB>
__global__ void __launch_bounds__(kThreads, 2) decode_mma_kernel(const DecodeArgs a) {
  constexpr int kKeyBytes = DK * 2, kValBytes = DV * 2, kStageBytes = stage_bytes<DK, DV>();
  constexpr int CK = DK / 8, CV = DV / 8;  // 16-byte pieces per row
  extern __shared__ __align__(128) uint8_t smem[];
  unsigned* prefix = reinterpret_cast<unsigned*>(smem + ring_bytes<DK, DV>());
  __shared__ float ms[kWarps][8 * NB], ls[kWarps][8 * NB];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // Pieces past dk / dv are never copied: they stay zero.
  for (int e = tid; e < ring_bytes<DK, DV>() / 16; e += kThreads) reinterpret_cast<uint4*>(smem)[e] = make_uint4(0, 0, 0, 0);
  pdl_wait();
  pdl_launch_dependents();
  tile_prefix(a, prefix);
  const int per_seq = a.Hkv * a.chunks;
  const long long total = static_cast<long long>(prefix[a.B]) * per_seq;
  const Run run{total, min(static_cast<long long>(gridDim.x), max(total, 1LL))};
  const long long cta = blockIdx.x;
  if (tid == 0) a.record[2 * cta] = -1;
  zero_empty(a, prefix, [&](long long at) { static_cast<__nv_bfloat16*>(a.o)[at] = __float2bfloat16_rn(0.f); });
  if (cta >= run.ctas || total == 0) return;
  const long long end = run.begin(cta + 1);
  long long at = run.begin(cta);
  int b = find_seq(a, prefix, per_seq, at);

  uint8_t* ring = smem + warp * kStages * kStageBytes;
  const uint32_t ring_addr = smem_u32(ring);
  const int kq = a.dk / 8, vq = a.dv / 8;  // real pieces per row
  const float c_scale = a.scale * kLog2e;
  const bool cap = a.softcap > 0.f, bias = a.slopes != nullptr;
  const float cap_a = a.softcap * kLog2e, cap_k = cap ? 2.f * c_scale / a.softcap : 0.f;
  const int g = lane >> 2, t4 = lane & 3;
  // Within a stage: this lane's first copy targets and its rows' addresses for
  // ldmatrix.  Stages and rows are multiples of 128 bytes, so the swizzle of a
  // later row or piece is an exclusive or on the address.
  const uint32_t k_dst = (lane / CK) * kKeyBytes + (((lane % CK) ^ (lane / CK)) * 16);
  const uint32_t v_dst = kStep * kKeyBytes + (lane / CV) * kValBytes + (((lane % CV) ^ (lane / CV)) * 16);
  const uint32_t k_src = ((lane & 7) + 8 * ((lane >> 3) & 1)) * kKeyBytes + (((lane >> 4) ^ (lane & 7)) * 16);
  const uint32_t v_src = ((lane & 7) + 8 * (lane >> 4)) * kValBytes + ((((lane >> 3) & 1) ^ (lane & 7)) * 16);
  const bool same = a.cache.ks_p == a.cache.vs_p && a.cache.ks_t == a.cache.vs_t;  // one offset serves both

  while (at < end) {
    const Piece pc = next_piece(a, prefix, per_seq, at, end, &b);
    const char* kbase = static_cast<const char*>(a.cache.k) + pc.hk * a.cache.ks_h * 2 + (lane % CK) * 16;
    const char* vbase = static_cast<const char*>(a.cache.v) + pc.hk * a.cache.vs_h * 2 + (lane % CV) * 16;

    // Q^T as the MMA's B operand: head g of each 8, elements 2 t4 and 2 t4 + 8 of each 16
    uint32_t qf[DK / 16][NB][2];
#pragma unroll
    for (int s = 0; s < DK / 16; ++s)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int hd = g + 8 * nb, d = 16 * s + 2 * t4 + 8 * r;
          uint32_t w = 0;
          if (hd < pc.heads && d < a.dk) {  // dk is even
            const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + pc.b * a.qs_b + (pc.h0 + hd) * a.qs_h + d;
            w = static_cast<uint32_t>(__bfloat16_as_ushort(q[0])) | (static_cast<uint32_t>(__bfloat16_as_ushort(q[1])) << 16);
          }
          qf[s][nb][r] = w;
        }
    // This thread's heads are 8 nb + 2 t4 and the one after.
    float slope[NB][2], m[NB][2], l[NB][2], o[DV / 16][NB][4];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int hd = 8 * nb + 2 * t4 + e;
        slope[nb][e] = bias && hd < pc.heads ? a.slopes[pc.h0 + hd] * kLog2e : 0.f;
        m[nb][e] = kNegInf;
        l[nb][e] = 0.f;
      }
#pragma unroll
      for (int d = 0; d < DV / 16; ++d)
#pragma unroll
        for (int r = 0; r < 4; ++r) o[d][nb][r] = 0.f;
    }

    // Lane x < 16 looks token x of a step up, one step before its copies are
    // issued: the byte offsets of its rows, or -1.
    const int base = pc.tile0 * kDecodeTile + warp * kStep;
    struct Rows {
      long long k, v;
    };
    auto lookup = [&](int step) {
      const int j = base + step * kDecodeTile + (lane & 15);
      Rows r{-1, -1};
      if (step < pc.tiles && j >= pc.lo && j < pc.hi) {
        int slot;
        const long long page = token_page(a, pc.b, j, &slot);
        if (page >= 0) {
          r.k = (page * a.cache.ks_p + slot * a.cache.ks_t) * 2;
          r.v = same ? r.k : (page * a.cache.vs_p + slot * a.cache.vs_t) * 2;
        }
      }
      return r;
    };
    unsigned live[kStages];  // bit x: token x of the stage's step exists
    auto issue = [&](int step, int stage, const Rows& rows) {
      const unsigned have = __ballot_sync(~0u, rows.k >= 0) & 0xffffu;
      if (step < pc.tiles) {
        const uint32_t kd = ring_addr + stage * kStageBytes + k_dst, vd = ring_addr + stage * kStageBytes + v_dst;
#pragma unroll
        for (int i = 0; i < kStep * CK / 32; ++i) {  // 32 / CK rows at a time
          const int r = i * (32 / CK) + lane / CK;
          const long long at = __shfl_sync(~0u, rows.k, r);
          const bool ok = (have >> r) & 1;
          // row r's pieces lie at piece ^ (r % 8)
          if (lane % CK < kq) cp_async16((kd + i * (32 / CK) * kKeyBytes) ^ ((i * (32 / CK) & 7) * 16), ok ? kbase + at : kbase, ok);
          if (CK == CV) {
            const long long to = same ? at : __shfl_sync(~0u, rows.v, r);
            if (lane % CV < vq) cp_async16((vd + i * (32 / CV) * kValBytes) ^ ((i * (32 / CV) & 7) * 16), ok ? vbase + to : vbase, ok);
          }
        }
        if (CK != CV) {
#pragma unroll
          for (int i = 0; i < kStep * CV / 32; ++i) {
            const int r = i * (32 / CV) + lane / CV;
            const long long to = __shfl_sync(~0u, rows.v, r);
            const bool ok = (have >> r) & 1;
            if (lane % CV < vq) cp_async16((vd + i * (32 / CV) * kValBytes) ^ ((i * (32 / CV) & 7) * 16), ok ? vbase + to : vbase, ok);
          }
        }
      }
      cp_async_commit();
      return have;
    };

#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) live[s] = issue(s, s, lookup(s));
    Rows rows = lookup(kStages - 1);
    int stage = 0;
    for (int step = 0; step < pc.tiles; ++step) {
      const int fill = stage == 0 ? kStages - 1 : stage - 1;  // the stage read in the last step
      __syncwarp();
      {
        const unsigned lv = issue(step + kStages - 1, fill, rows);
#pragma unroll
        for (int s = 0; s < kStages; ++s)
          if (s == fill) live[s] = lv;
      }
      rows = lookup(step + kStages);
      cp_async_wait<kStages - 1>();
      __syncwarp();
      unsigned lv = 0;
#pragma unroll
      for (int s = 0; s < kStages; ++s)
        if (s == stage) lv = live[s];
      const uint32_t ks = ring_addr + stage * kStageBytes, vs = ks + kStep * kKeyBytes;
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
      // x = log2(e) * score
      const int j0 = base + step * kDecodeTile;
      const float dist = static_cast<float>(pc.len - 1 - j0 - g);
      bool grow = false;
      float mx[NB][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float x = s[nb][r];
          if (cap) {
            // cap * tanh(s / cap) = cap - 2 cap / (1 + e^(2 s / cap))
            float den;
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(den) : "f"(1.f + exp2_approx(x * cap_k)));
            x = fmaf(-2.f * cap_a, den, cap_a);
          } else {
            x *= c_scale;
          }
          if (bias) x = fmaf(-slope[nb][r & 1], dist - 8.f * (r >> 1), x);
          if (lv != 0xffffu && !((lv >> (g + 8 * (r >> 1))) & 1)) x = kNegInf;
          s[nb][r] = x;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float y = fmaxf(s[nb][e], s[nb][2 + e]);
          y = fmaxf(y, __shfl_xor_sync(~0u, y, 4));
          y = fmaxf(y, __shfl_xor_sync(~0u, y, 8));
          y = fmaxf(y, __shfl_xor_sync(~0u, y, 16));
          mx[nb][e] = y;
          grow |= y > m[nb][e] + kGrowth;
        }
      }
      if (__any_sync(~0u, grow)) {
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
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    cp_async_wait<0>();
    __syncthreads();  // every warp is through with its ring: it now takes the results [warp][heads][DV]
    float* res = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float y = l[nb][e];
        y += __shfl_xor_sync(~0u, y, 4);
        y += __shfl_xor_sync(~0u, y, 8);
        y += __shfl_xor_sync(~0u, y, 16);
        const int hd = 8 * nb + 2 * t4 + e;
        if (g == 0) ms[warp][hd] = m[nb][e], ls[warp][hd] = y;
        if (hd < pc.heads)
#pragma unroll
          for (int d = 0; d < DV / 16; ++d) {
            res[(warp * pc.heads + hd) * DV + 16 * d + g] = o[d][nb][e];
            res[(warp * pc.heads + hd) * DV + 16 * d + g + 8] = o[d][nb][2 + e];
          }
      }
    __syncthreads();
    float* part = a.part + (2 * cta + (pc.starts ? 1 : 0)) * part_floats(a.item_heads, a.dv);
    const bool whole = pc.starts && pc.ends;
    for (int e = tid; e < pc.heads * DV; e += kThreads) {
      const int hd = e / DV, d = e % DV;
      if (d >= a.dv) continue;
      float mm = kNegInf;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, ms[w][hd]);
      const float mu = mm == kNegInf ? 0.f : mm;
      float sum = 0.f, ll = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = exp2_approx(ms[w][hd] - mu);
        sum = fmaf(f, res[(w * pc.heads + hd) * DV + d], sum);
        ll = fmaf(f, ls[w][hd], ll);
      }
      if (whole) {
        static_cast<__nv_bfloat16*>(a.o)[pc.b * a.os_b + (pc.h0 + hd) * a.os_h + d] = __float2bfloat16_rn(ll == 0.f ? 0.f : sum / ll);
      } else {
        part[2 * a.item_heads + hd * a.dv + d] = sum;
        if (d == 0) part[hd] = mm, part[a.item_heads + hd] = ll;
      }
    }
    if (!whole && pc.starts && tid == 0) note_item(a, run, pc, per_seq, cta);
    at += pc.tiles;
    __syncthreads();
    // the pieces past dk / dv are zero again
    if (at < end && (kq < CK || vq < CV)) {
      for (int e = tid; e < ring_bytes<DK, DV>() / 16; e += kThreads) reinterpret_cast<uint4*>(smem)[e] = make_uint4(0, 0, 0, 0);
      __syncthreads();
    }
  }
}

template <int DK, int DV, int NB>
cudaError_t launch_one(const DecodeArgs& a, cudaStream_t s) {
  const size_t smem = ring_bytes<DK, DV>() + sizeof(unsigned) * (a.B + 1);
  const cudaError_t e = smem_attr_once<decode_mma_kernel<DK, DV, NB>>(smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(decode_mma_kernel<DK, DV, NB>, dim3(a.ctas), dim3(kThreads), smem, s, a);
}

template <int DK, int DV>
cudaError_t launch_dims(const DecodeArgs& a, cudaStream_t s) {
  return a.item_heads <= 8 ? launch_one<DK, DV, 1>(a, s) : launch_one<DK, DV, 2>(a, s);
}

}  // namespace

cudaError_t launch_decode_mma(const DecodeArgs& a, cudaStream_t s) {
  if (a.dk <= 64) return a.dv <= 64 ? launch_dims<64, 64>(a, s) : launch_dims<64, 128>(a, s);
  return a.dv <= 64 ? launch_dims<128, 64>(a, s) : launch_dims<128, 128>(a, s);
}

}  // namespace cb
