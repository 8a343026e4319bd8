// The streaming attention kernel for few queries per key head, over keys and
// values whose rows are whole 16-byte pieces.  A policy C does the arithmetic
// (decode_mma.cu: bf16 by warp-level MMAs; decode_fma.cu: fp32 by FMAs) for
// one of two sources:
//  - a paged cache and one new token per sequence (cb_attention_decode): an
//    item's columns are query heads that share a key head;
//  - contiguous rows and short query sequences (cb_attention, C::kRows): an
//    item's columns are (query, head) pairs that share a key head, each with
//    its own visible keys.
//
// Bound by HBM: (dk + dv) * sizeof(element) bytes per cached token and key
// head, read once.  A CTA's four warps walk a piece of one item together: each
// takes its own kStep tokens of every kWarps * kStep through its own ring of
// cp.async copies and keeps its own maximum, sum and O, so nothing synchronises
// inside a piece; the four are joined when it ends.
//
// Two ways to deal items (decode_common.cuh):
//  - Runs: equal runs of tiles over one wave of CTAs; items cut by a run's end
//    go through the workspace and a join kernel.
//  - Whole items, for caches small enough that a CTA walks at most 16 tiles
//    and for contiguous rows: a cluster of a.split CTAs per item, joined
//    through distributed shared memory.  One launch, no prefix over the
//    lengths: one sequence of 421 tokens takes 4.7 us where runs and their join
//    take 9.4, 64 of 200 to 500 tokens (8 key heads of 128) 25 and 33; from
//    about 30 tiles per CTA on runs are faster (32 sequences of 100 to 2000
//    tokens: 37, whole 41).
#pragma once

#include "decode_common.cuh"
#include "launch_util.h"
#include "ptx.cuh"

namespace cb {

constexpr int kDecodeWarps = 4, kDecodeThreads = kDecodeWarps * 32;
constexpr float kDecodeGrowth = 8.f;  // rescale O when a maximum grew by more (log2)

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// log2(e) * score of a dot product, as the decode kernels evaluate it. Capped: cap tanh(y), y = s / cap, exact to a
// few 2^-24 of the score however far below its cap it lies:
//   |y| <= 0.8  s Q(y^2), Q the minimax fit of tanh(y) / y there, of degree 5 in y^2 (relative error 6e-8);
//   beyond      cap - 2 cap / (1 + e^(2 |y|)) with the score's sign: what is subtracted is at most 0.34 of the cap.
// (The second form alone loses a few 2^-24 of the cap, all of a score that is small enough beside it.)
struct DecodeScore {
  float c_scale, cap_a, cap_in, cap_k;
  bool cap;
  __device__ __forceinline__ explicit DecodeScore(const DecodeArgs& a) {
    c_scale = a.scale * kLog2e;
    cap = a.softcap > 0.f;
    cap_a = a.softcap * kLog2e;
    cap_in = cap ? a.scale / a.softcap : 0.f;
    cap_k = 2.f * kLog2e * cap_in;
  }
  static constexpr float kNear = 0.8f;
  __device__ __forceinline__ float near(float dot) const {
    const float y = dot * cap_in, z = y * y;
    float g = fmaf(z, -0.00435529975220561f, 0.01909330114722252f);
    g = fmaf(z, g, -0.05311431735754013f);
    g = fmaf(z, g, 0.13321048021316528f);
    g = fmaf(z, g, -0.3333267569541931f);
    g = fmaf(z, g, 0.9999999403953552f);
    return dot * c_scale * g;
  }
  __device__ __forceinline__ float far(float dot) const {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + exp2_approx(fabsf(dot) * cap_k)));
    return copysignf(fmaf(-2.f * cap_a, r, cap_a), dot);
  }
  // In place, by a whole warp: the second form only where one of its scores needs it.
  template <int M, int N>
  __device__ __forceinline__ void operator()(float (&s)[M][N]) const {
    if (!cap) {
#pragma unroll
      for (int i = 0; i < M; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) s[i][j] *= c_scale;
      return;
    }
    float big = 0.f;
#pragma unroll
    for (int i = 0; i < M; ++i)
#pragma unroll
      for (int j = 0; j < N; ++j) big = fmaxf(big, fabsf(s[i][j]));
    const bool some = __any_sync(~0u, big * cap_in > kNear);
#pragma unroll
    for (int i = 0; i < M; ++i)
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float dot = s[i][j];
        s[i][j] = near(dot);
        if (some && !(fabsf(dot) * cap_in <= kNear)) s[i][j] = far(dot);
      }
  }
};

// Where column hd of an item comes from and goes to.
template <bool ROWS, typename T>
__device__ __forceinline__ const T* query_row(const DecodeArgs& a, const AttnArgs& rw, const Piece& pc, int hd) {
  if constexpr (ROWS) {
    const int r = pc.h0 + hd;
    return static_cast<const T*>(rw.q) + pc.b * rw.qs_b + r / a.group * rw.qs_l + (pc.hk * a.group + r % a.group) * rw.qs_h;
  }
  return static_cast<const T*>(a.q) + pc.b * a.qs_b + (pc.h0 + hd) * a.qs_h;
}
template <bool ROWS, typename T>
__device__ __forceinline__ T* out_row(const DecodeArgs& a, const AttnArgs& rw, const Piece& pc, int hd) {
  if constexpr (ROWS) {
    const int r = pc.h0 + hd;
    return static_cast<T*>(rw.o) + pc.b * rw.os_b + r / a.group * rw.os_l + (pc.hk * a.group + r % a.group) * rw.os_h;
  }
  return static_cast<T*>(a.o) + pc.b * a.os_b + (pc.h0 + hd) * a.os_h;
}
__device__ __forceinline__ float slope_of(const DecodeArgs& a, const AttnArgs& rw, const Piece& pc, int hd, bool rows) {
  const float* slopes = rows ? rw.slopes : a.slopes;
  if (!slopes || hd >= pc.heads) return 0.f;
  return slopes[rows ? pc.hk * a.group + (pc.h0 + hd) % a.group : pc.h0 + hd] * kLog2e;
}
// What a row query sees: keys [0, hi) of its document; it stands at `at`.
struct RowRule {
  int hi, at, doc;
};
__device__ __forceinline__ RowRule row_rule(const DecodeArgs& a, const AttnArgs& rw, const Piece& pc, int hd) {
  RowRule r{0, 0, -2};
  if (hd >= pc.heads) return r;
  const int i = (pc.h0 + hd) / a.group;
  r.hi = row_end(rw, seq_rule(rw, pc.b), i);
  r.at = i + rw.q_offset;
  r.doc = rw.doc_q ? rw.doc_q[static_cast<long long>(pc.b) * rw.Lq + i] : -1;  // without documents a key's is -1 too
  if (rw.doc_q && r.doc < 0) r.hi = 0;
  return r;
}

template <class C>
constexpr int decode_ring_bytes() {  // also holds the results when a piece ends
  return kDecodeWarps * C::kStages * C::kStep * (C::DK + C::DV) * static_cast<int>(sizeof(typename C::T));
}
template <class C>
constexpr int decode_part_offset() {  // floats: the four warps' results, then the CTA's
  return kDecodeWarps * C::kHeads * C::DV;
}

template <class C, bool WHOLE>
__global__ void __launch_bounds__(kDecodeThreads, decode_ctas_per_sm(C::DK, C::DV, sizeof(typename C::T) == 2, C::kHeads, 0))
    decode_stream_kernel(const DecodeArgs a, const AttnArgs rw) {
  using T = typename C::T;
  constexpr int DK = C::DK, DV = C::DV, kStep = C::kStep, kStages = C::kStages, kEl = static_cast<int>(sizeof(T));
  constexpr int kKeyBytes = DK * kEl, kValBytes = DV * kEl, kStageBytes = kStep * (kKeyBytes + kValBytes);
  constexpr int CK = kKeyBytes / 16, CV = kValBytes / 16;  // 16-byte pieces per row
  constexpr int RK = 32 / CK, RV = 32 / CV;                // rows per warp-wide copy
  static_assert(decode_ring_bytes<C>() >= 4 * (decode_part_offset<C>() + C::kHeads * DV), "results fit the ring");
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* after = smem + decode_ring_bytes<C>();
  __shared__ float ms[kDecodeWarps][C::kHeads], ls[kDecodeWarps][C::kHeads];
  __shared__ float part_m[C::kHeads], part_l[C::kHeads];
  __shared__ int odd[C::kHeads];  // contiguous rows: columns with a result that is not finite

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int kq = a.dk * kEl / 16, vq = a.dv * kEl / 16;  // real pieces per row
  const bool padded = kq < CK || vq < CV;
  auto clear = [&] {  // pieces past dk / dv are never copied: they stay zero
    for (int e = tid; e < decode_ring_bytes<C>() / 16; e += kDecodeThreads) reinterpret_cast<uint4*>(smem)[e] = make_uint4(0, 0, 0, 0);
  };
  if (padded) clear();
  pdl_wait();
  pdl_launch_dependents();
  const int per_seq = a.Hkv * a.chunks;
  unsigned* prefix = reinterpret_cast<unsigned*>(after + C::kExtra);
  long long at = 0, end = 1, cta = blockIdx.x;
  Run run{1, 1};
  int b = 0;
  if constexpr (!WHOLE) {
    tile_prefix(a, prefix);
    const long long total = static_cast<long long>(prefix[a.B]) * per_seq;
    run = Run{total, min(static_cast<long long>(gridDim.x), max(total, 1LL))};
    if (tid == 0) a.record[2 * cta] = -1;
    zero_empty(a, prefix, [&](long long i) { static_cast<T*>(a.o)[i] = from_f32<T>(0.f); });
    if (cta >= run.ctas || total == 0) return;
    at = run.begin(cta);
    end = run.begin(cta + 1);
    b = find_seq(a, prefix, per_seq, at);
  } else {
    __syncthreads();
  }

  // Within a stage: this lane's first copy targets.  Row r's pieces lie at
  // piece ^ swizzle(r), and swizzle is linear over exclusive or, so a later
  // row's address differs by a constant and an exclusive or.
  uint8_t* ring = smem + warp * kStages * kStageBytes;
  const uint32_t ring_addr = smem_u32(ring);
  const uint32_t k_dst = (lane / CK) * kKeyBytes + (((lane % CK) ^ C::swizzle(lane / CK)) * 16);
  const uint32_t v_dst = kStep * kKeyBytes + (lane / CV) * kValBytes + (((lane % CV) ^ C::swizzle(lane / CV)) * 16);
  const bool same = a.cache.ks_p == a.cache.vs_p && a.cache.ks_t == a.cache.vs_t;  // one offset serves both

  // Steps as short as they can be, but for runs of bf16 tokens, which HBM bounds: there warps that wait less
  // for themselves run further apart, and memory is the slower for it (8 sequences of up to 131072 tokens 483 us,
  // with eager steps 510; 8 of 300 to 1700, whole: 13.7 and 13.2; two fp32 sequences of 93000: 249 and 222).
  constexpr bool kEager = WHOLE || sizeof(T) == 4;
  // from a lane's token to its next one, without a division per step
  const int adv_pg = C::kRows ? 0 : kDecodeWarps * kStep / a.cache.page_size, adv_slot = kDecodeWarps * kStep - adv_pg * a.cache.page_size;

  while (at < end) {
    static_assert(WHOLE || !C::kRows, "contiguous rows are dealt as whole items");
    Piece pc;
    if constexpr (C::kRows) pc = rows_piece(a, rw);
    else if constexpr (WHOLE) pc = whole_piece(a, per_seq);
    else pc = next_piece(a, prefix, per_seq, at, end, &b);
    const char* kbase = static_cast<const char*>(a.cache.k) + pc.hk * a.cache.ks_h * kEl + (lane % CK) * 16;
    const char* vbase = static_cast<const char*>(a.cache.v) + pc.hk * a.cache.vs_h * kEl + (lane % CV) * 16;

    // Lanes below kStep look the step's tokens up, one step before their copies
    // are issued: the byte offsets of the rows, or -1.
    const int base = pc.tile0 * kDecodeTile + warp * kStep;
    const int steps = pc.tiles * (kDecodeTile / (kDecodeWarps * kStep));
    struct Rows {
      long long k, v;
      int doc;  // contiguous rows: the key's document
    };
    // j is unsigned: a token looked up past the piece's end may be past 2^31
    unsigned j = base + lane % kStep;
    int pg = C::kRows ? 0 : static_cast<int>(j) / a.cache.page_size, slot = C::kRows ? 0 : static_cast<int>(j) - pg * a.cache.page_size;
    auto lookup = [&](int step) {  // once for each step, in order
      Rows r{-1, -1, -1};
      if (step < steps && j >= static_cast<unsigned>(pc.lo) && j < static_cast<unsigned>(pc.hi)) {
        if constexpr (C::kRows) {
          r.k = (pc.b * a.cache.ks_p + j * a.cache.ks_t) * kEl;
          r.v = (pc.b * a.cache.vs_p + j * a.cache.vs_t) * kEl;
          if (rw.doc_k) r.doc = rw.doc_k[static_cast<long long>(pc.b) * rw.Lk + j];
        } else {
          if (!kEager) pg = static_cast<int>(j) / a.cache.page_size, slot = static_cast<int>(j) - pg * a.cache.page_size;
          const long long page = checked_page(a, pc.b, pg);
          if (page >= 0) {
            r.k = (page * a.cache.ks_p + slot * a.cache.ks_t) * kEl;
            r.v = same ? r.k : (page * a.cache.vs_p + slot * a.cache.vs_t) * kEl;
          }
        }
      }
      j += kDecodeWarps * kStep;
      if (kEager && !C::kRows) {
        pg += adv_pg, slot += adv_slot;
        if (slot >= a.cache.page_size) slot -= a.cache.page_size, ++pg;
      }
      return r;
    };
    constexpr unsigned kAll = kStep == 32 ? ~0u : (1u << kStep) - 1;
    unsigned live[kStages];  // bit x: token x of the stage's step exists
    int docs[kStages];
    auto issue = [&](int step, int stage, const Rows& rows) {
      const unsigned have = __ballot_sync(~0u, rows.k >= 0) & kAll;
      if (step < steps) {
        const uint32_t kd = ring_addr + stage * kStageBytes + k_dst, vd = ring_addr + stage * kStageBytes + v_dst;
#pragma unroll
        for (int i = 0; i < kStep / RK; ++i) {
          const int r = i * RK + lane / CK;
          const long long off = __shfl_sync(~0u, rows.k, r);
          const bool ok = (have >> r) & 1;
          if (lane % CK < kq) cp_async16((kd + i * RK * kKeyBytes) ^ (C::swizzle(i * RK) * 16), ok ? kbase + off : kbase, ok);
          if (CK == CV) {
            const long long to = same ? off : __shfl_sync(~0u, rows.v, r);
            if (lane % CV < vq) cp_async16((vd + i * RV * kValBytes) ^ (C::swizzle(i * RV) * 16), ok ? vbase + to : vbase, ok);
          }
        }
        if (CK != CV) {
#pragma unroll
          for (int i = 0; i < kStep / RV; ++i) {
            const int r = i * RV + lane / CV;
            const long long to = __shfl_sync(~0u, rows.v, r);
            const bool ok = (have >> r) & 1;
            if (lane % CV < vq) cp_async16((vd + i * RV * kValBytes) ^ (C::swizzle(i * RV) * 16), ok ? vbase + to : vbase, ok);
          }
        }
      }
      cp_async_commit();
      return have;
    };

#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) {
      const Rows r = lookup(s);
      live[s] = issue(s, s, r);
      docs[s] = r.doc;
    }
    C c(a, rw, pc, after);  // the queries are read while the first tokens come
    Rows rows = lookup(kStages - 1);
    int stage = 0;
    for (int step = 0; step < steps; ++step) {
      const int fill = stage == 0 ? kStages - 1 : stage - 1;  // the stage read in the last step
      __syncwarp();
      {
        const unsigned lv = issue(step + kStages - 1, fill, rows);
#pragma unroll
        for (int s = 0; s < kStages; ++s)
          if (s == fill) live[s] = lv, docs[s] = rows.doc;
      }
      rows = lookup(step + kStages);
      cp_async_wait<kStages - 1>();
      __syncwarp();
      unsigned lv = 0;
      int doc = 0;
#pragma unroll
      for (int s = 0; s < kStages; ++s)
        if (s == stage) lv = live[s], doc = docs[s];
      const uint32_t ks = ring_addr + stage * kStageBytes;
      // a decode query stands pc.len - 1 - j before key j; a row query knows its own place
      const int j0 = base + step * (kDecodeWarps * kStep);
      c.template step<kEager>(ks, ks + kStep * kKeyBytes, lv, C::kRows ? j0 : pc.len - 1 - j0, doc);
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    cp_async_wait<0>();
    __syncthreads();  // every warp is through with its ring: it now takes the results [warp][heads][DV]
    float* res = reinterpret_cast<float*>(smem);
    c.store(res + warp * pc.heads * DV, ms[warp], ls[warp]);
    __syncthreads();
    // The four warps' results as one: into the output, the workspace, or (whole
    // items of a cluster) this CTA's part.
    float* part_s = res + decode_part_offset<C>();
    float* part = WHOLE ? nullptr : a.part + (2 * cta + (pc.starts ? 1 : 0)) * part_floats(a.item_heads, a.dv);
    const bool out = pc.starts && pc.ends;
    if (C::kRows && tid < C::kHeads) odd[tid] = 0;
    if (tid < pc.heads) {
      float mm = kNegInf, ll = 0.f, f[kDecodeWarps];
#pragma unroll
      for (int w = 0; w < kDecodeWarps; ++w) mm = fmaxf(mm, ms[w][tid]);
      const float mu = mm == kNegInf ? 0.f : mm;
#pragma unroll
      for (int w = 0; w < kDecodeWarps; ++w) {
        f[w] = exp2_approx(ms[w][tid] - mu);
        ll = fmaf(f[w], ls[w][tid], ll);
      }
      const float inv = !out ? 1.f : ll == 0.f ? 0.f : 1.f / ll;
#pragma unroll
      for (int w = 0; w < kDecodeWarps; ++w) ms[w][tid] = f[w] * inv;
      if constexpr (WHOLE) part_m[tid] = mm, part_l[tid] = ll;
      else if (!out) part[tid] = mm, part[a.item_heads + tid] = ll;
    }
    __syncthreads();
    bool bad = false;
    auto put = [&](int hd, int d, float y, float sum) {
      out_row<C::kRows, T>(a, rw, pc, hd)[d] = from_f32<T>(y);
      if (C::kRows && !(y * 0.f == 0.f) && sum == sum) bad = true, odd[hd] = 1;
    };
    for (int e = tid; e < pc.heads * DV; e += kDecodeThreads) {
      const int hd = e / DV, d = e % DV;
      if (d >= a.dv) continue;
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kDecodeWarps; ++w) sum = fmaf(ms[w][hd], res[(w * pc.heads + hd) * DV + d], sum);
      if (out) put(hd, d, sum, C::kRows ? part_l[hd] : 0.f);
      else if constexpr (WHOLE) part_s[hd * DV + d] = sum;
      else part[2 * a.item_heads + hd * a.dv + d] = sum;
    }
    if constexpr (WHOLE) {
      if (a.split > 1) {  // the cluster's CTAs share the item: each joins every a.split-th value of all
        cluster_sync();
        for (int e = tid * a.split + static_cast<int>(cluster_ctarank()); e < pc.heads * DV; e += kDecodeThreads * a.split) {
          const int hd = e / DV, d = e % DV;
          if (d >= a.dv) continue;
          float m[8], mm = kNegInf, sum = 0.f, ll = 0.f;
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            m[r] = r < a.split ? ld_cluster_f32(map_shared_rank(smem_u32(part_m + hd), r)) : kNegInf;
            mm = fmaxf(mm, m[r]);
          }
          const float mu = mm == kNegInf ? 0.f : mm;
#pragma unroll
          for (int r = 0; r < 8; ++r)
            if (r < a.split) {
              const float f = exp2_approx(m[r] - mu);
              sum = fmaf(f, ld_cluster_f32(map_shared_rank(smem_u32(part_s + e), r)), sum);
              ll = fmaf(f, ld_cluster_f32(map_shared_rank(smem_u32(part_l + hd), r)), ll);
            }
          put(hd, d, ll == 0.f ? 0.f : sum / ll, ll);
        }
        cluster_sync();  // the parts are read before any CTA leaves
      }
      if constexpr (C::kRows) {
        // Rows that met a hidden value that is not finite: again, key by key. A column per lane.
        if (__syncthreads_or(bad)) {
          const bool mine = lane < pc.heads && odd[lane];
          const RowRule r = row_rule(a, rw, pc, lane);
          const unsigned again = rows_to_redo<T, true>(rw, pc.b, pc.hk, pc.hi, mine, r.hi, r.doc, 1.f);
          for (int hd = warp; hd < pc.heads; hd += kDecodeWarps)
            if ((again >> hd) & 1) attn_row<T, true>(rw, pc.b, pc.hk * a.group + (pc.h0 + hd) % a.group, (pc.h0 + hd) / a.group);
        }
      }
      return;
    }
    if (!out && pc.starts && tid == 0) note_item(a, run, pc, per_seq, cta);
    at += pc.dealt;
    __syncthreads();
    if (at < end && padded) {
      clear();
      __syncthreads();
    }
  }
}

template <class C>
cudaError_t launch_whole(const DecodeArgs& a, const AttnArgs& rw, long long ctas, cudaStream_t s) {
  const size_t smem = decode_ring_bytes<C>() + C::kExtra;
  const cudaError_t e = smem_attr_once<decode_stream_kernel<C, true>>(smem);
  if (e != cudaSuccess) return e;
  if (ctas >= (1LL << 31)) return cudaErrorInvalidConfiguration;
  const dim3 grid(static_cast<unsigned>(ctas));
  if (a.split == 1) return launch_pdl(decode_stream_kernel<C, true>, grid, dim3(kDecodeThreads), smem, s, a, rw);
  return launch_pdl_cluster(decode_stream_kernel<C, true>, grid, dim3(kDecodeThreads), smem, s, a.split, a, rw);
}

template <class C>
cudaError_t launch_decode_stream(const DecodeArgs& a, cudaStream_t s) {
  const AttnArgs none{};
  if (a.split) return launch_whole<C>(a, none, static_cast<long long>(a.B) * a.Hkv * a.chunks * a.split, s);
  const size_t smem = decode_ring_bytes<C>() + C::kExtra + sizeof(unsigned) * (a.B + 1);
  const cudaError_t e = smem_attr_once<decode_stream_kernel<C, false>>(smem);
  if (e != cudaSuccess) return e;
  // After the kernel before it, not among its CTAs: this wave fills the SMs exactly, and CTAs that came while others
  // still held some of them would be placed unevenly (104 sequences of about 2000 fp32 tokens, 2 heads: 65 us, so 45).
  return launch_serial(decode_stream_kernel<C, false>, dim3(a.ctas), dim3(kDecodeThreads), smem, s, a, none);
}

}  // namespace cb
