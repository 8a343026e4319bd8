// Attention on the tensor cores: bf16 views of whole 16-byte pieces.
//
// One CTA owns 256 queries of one head as two tiles t of 128 and walks the
// visible key tiles of 128 with a running maximum and sum per query:
//   S_t = Q_t K^T        tcgen05.mma, both operands in shared memory (TMA, 128-byte swizzle),
//                        fp32 accumulator in 128 TMEM columns
//   P_t = 2^(x - m)      x = log2(e) * score, by one warpgroup per tile, a thread per query:
//                        tcgen05.ld of its 128 scores, P rounded to bf16 and stored over S_t
//   O_t += P_t V         tcgen05.mma with A = P_t from TMEM and B = V as it lies (rows of keys:
//                        the MN-major operand), O_t in up to 128 further columns
// The tiles take turns: while one warpgroup computes P of tile 0, the tensor
// cores work on tile 1.  One thread issues, in the order
//   PV_0(n), QK_0(n+1), PV_1(n), QK_1(n+1),
// so S_t is overwritten only by an MMA issued after the one that reads P_t, and
// the commit after QK_t(n+1) also covers PV_t(n): once a warpgroup sees S_t(n+1)
// it may rescale O_t without another barrier.
//
// O is rescaled only when a query's maximum has grown by more than 2^8 since
// the last time; until then weights are relative to the older maximum (at most
// 2^8, exact in fp32 and of the same relative precision in bf16) and l and O
// agree on it.  P is rounded to bf16 for the second product (2^-9 relative at
// most to nearest, independent from key to key); l sums the unrounded weights.
//
// Key tiles no query of the CTA sees are never loaded: a list of the tiles to
// visit, with each query tile's state (skip, full, masked), is made first.
#include "attention_common.cuh"
#include "launch_util.h"
#include "ptx.cuh"

namespace cb {

namespace {

constexpr int kTile = 128;          // queries per tile, keys per tile
constexpr int kSlab = 128 * 128;    // bytes of 128 rows x 64 bf16
// Two softmax warpgroups and a third with the copy warp, the MMA warp and two
// idle ones: at launch every thread holds 168 registers (the most for 12
// warps), then the third warpgroup hands its own to the other two, whose
// threads keep 128 scores each: 2 * 128 * 224 + 128 * 56 = 384 * 168.
constexpr int kThreads = 384;
constexpr int kSoftmaxRegs = 224, kOtherRegs = 56;
static_assert(256 * kSoftmaxRegs + 128 * kOtherRegs <= kThreads * 168, "registers of the launch");
constexpr int kCopyWarp = 8, kMmaWarp = 9;
constexpr float kGrowth = 8.f;      // rescale when the maximum grew by more (log2)

__device__ __forceinline__ void tmem_ld_x32f(uint32_t taddr, float* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]),
        "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]),
        "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_x32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// D[tmem] (+)= A[tmem] * B[smem], kind::f16 with bf16 operands: A row i in
// lane i, two K elements per column.
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Shared-memory descriptor of an MN-major operand: rows of K, each 64
// elements (128 bytes, swizzled) of N; the next 64 elements of N one slab
// further (leading byte offset), the next 8 rows of K 1024 bytes further
// (stride byte offset).
__device__ __forceinline__ uint64_t mnmajor_desc(uint32_t saddr) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(kSlab >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

enum : uint32_t { kSkip = 0, kFull = 1, kMasked = 2 };

template <int SK, int SV>
struct Shape {
  static constexpr int kSlot = (SK > SV ? SK : SV) * kSlab;  // one ring slot: a K or a V tile
  static constexpr int kStages = SK == 2 || SV == 2 ? 4 : 8;
  static constexpr int kQ = 2 * SK * kSlab;
  static constexpr int kFixed = kQ + kStages * kSlot + 8 * kTile * 4 /* doc ids */ + 512 /* barriers */ + 1024 /* alignment */;
};

template <int SK, int SV>
__global__ void __launch_bounds__(kThreads, 1)
attn_tc_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
               const __grid_constant__ CUtensorMap vmap, const AttnArgs a, int q_tiles) {
  using SH = Shape<SK, SV>;
  constexpr int NS = SH::kStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sKV = smem + SH::kQ;
  int* doc_buf = reinterpret_cast<int*>(sKV + NS * SH::kSlot);  // [8 warps][128]
  uint64_t* q_full = reinterpret_cast<uint64_t*>(doc_buf + 8 * kTile);
  uint64_t* kv_full = q_full + 2;
  uint64_t* kv_empty = kv_full + NS;
  uint64_t* s_full = kv_empty + NS;
  uint64_t* p_ready = s_full + 2;
  uint64_t* o_full = p_ready + 2;
  uint64_t* v_tail = o_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(v_tail + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* shared_n = reinterpret_cast<int*>(tmem_slot + 2);  // tiles in the list
  int* doc_range = shared_n + 1;                          // per query tile: min, max, any padding
  uint32_t* list = reinterpret_cast<uint32_t*>(reinterpret_cast<uint8_t*>(q_full) + 512);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(&q_full[t], 1);
      mbar_init(&s_full[t], 1);
      mbar_init(&p_ready[t], 4);
      mbar_init(&o_full[t], 1);
      doc_range[3 * t] = 0x7fffffff, doc_range[3 * t + 1] = -1, doc_range[3 * t + 2] = 0;
    }
    for (int s = 0; s < NS; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 1);
    }
    mbar_init(v_tail, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  pdl_launch_dependents();
  pdl_wait();
  const uint32_t tmem = *tmem_slot;
  const Watchdog wd{a.err, abort_flag, a.timeout_ns};

  // Last query tiles first: under a causal mask they are the longest.
  const int heads = a.B * a.Hq;
  const int qt = q_tiles - 1 - static_cast<int>(blockIdx.x / heads);
  const int bh = blockIdx.x % heads, b = bh / a.Hq, h = bh % a.Hq, hk = h / a.group;
  const int i0 = qt * 2 * kTile;
  const SeqRule rule = seq_rule(a, b);
  const bool docs = a.doc_k != nullptr;
  const int* doc_k = docs ? a.doc_k + static_cast<long long>(b) * a.Lk : nullptr;

  // ------------------------------------------------------------ the list
  int my_row = 0, my_doc = 0, my_hi = 0;  // warpgroups: this thread's query
  if (warp < 8) {
    my_row = i0 + threadIdx.x;
    if (my_row < a.Lq) {
      my_hi = row_end(a, rule, my_row);
      if (docs) my_doc = a.doc_q[static_cast<long long>(b) * a.Lq + my_row];
      if (my_doc < 0) my_hi = 0;
    }
    if (docs) {
      const int t = warp >> 2;
      const bool row = my_row < a.Lq;
      const int lo = __reduce_min_sync(~0u, row && my_doc >= 0 ? my_doc : 0x7fffffff);
      const int hi = __reduce_max_sync(~0u, row && my_doc >= 0 ? my_doc : -1);
      const bool pad = __any_sync(~0u, row && my_doc < 0);
      if (lane == 0) {
        atomicMin(&doc_range[3 * t], lo);
        atomicMax(&doc_range[3 * t + 1], hi);
        if (pad) doc_range[3 * t + 2] = 1;
      }
    }
  }
  int hi_lo[2], hi_hi[2];  // per query tile: keys that all / some of its queries see, before documents
  for (int t = 0; t < 2; ++t) {
    const int r0 = i0 + t * kTile, r1 = min(a.Lq, r0 + kTile) - 1;
    hi_lo[t] = r0 <= r1 ? row_end(a, rule, r0) : 0;
    hi_hi[t] = r0 <= r1 ? row_end(a, rule, r1) : 0;
  }
  const int all_tiles = (max(hi_hi[0], hi_hi[1]) + kTile - 1) / kTile;
  if (docs) __syncthreads();
  if (!docs) {
    for (int n = threadIdx.x; n < all_tiles; n += kThreads) {
      uint32_t e = n << 4;
      for (int t = 0; t < 2; ++t)
        e |= (n * kTile >= hi_hi[t] ? kSkip : (n + 1) * kTile <= hi_lo[t] ? kFull : kMasked) << (2 * t);
      list[n] = e;
    }
    if (threadIdx.x == 0) *shared_n = all_tiles;
  } else {
    for (int n = warp; n < all_tiles; n += kThreads / 32) {
      int lo = 0x7fffffff, hi = -0x7fffffff;
      for (int c = lane; c < kTile; c += 32) {
        const int j = n * kTile + c;
        if (j < rule.kv) lo = min(lo, doc_k[j]), hi = max(hi, doc_k[j]);
      }
      lo = __reduce_min_sync(~0u, lo);
      hi = __reduce_max_sync(~0u, hi);
      uint32_t e = n << 4;
      for (int t = 0; t < 2; ++t) {
        const int dlo = doc_range[3 * t], dhi = doc_range[3 * t + 1];
        uint32_t st = n * kTile >= hi_hi[t] || hi < dlo || lo > dhi ? kSkip : kMasked;
        if (st == kMasked && lo == hi && dlo == dhi && lo == dlo && !doc_range[3 * t + 2] && (n + 1) * kTile <= hi_lo[t])
          st = kFull;
        e |= st << (2 * t);
      }
      if (lane == 0) list[n] = e;
    }
    __syncthreads();
    if (warp == 0) {  // drop the tiles no query sees
      int kept = 0;
      for (int n0 = 0; n0 < all_tiles; n0 += 32) {
        const uint32_t e = n0 + lane < all_tiles ? list[n0 + lane] : 0;
        const unsigned keep = __ballot_sync(~0u, (e & 15u) != 0);
        __syncwarp();
        if (e & 15u) list[kept + __popc(keep & ((1u << lane) - 1))] = e;
        kept += __popc(keep);
        __syncwarp();
      }
      if (lane == 0) *shared_n = kept;
    }
  }
  __syncthreads();
  const int N = *shared_n;
  // A last tile that holds keys past kv_len: their values, whatever they are, become zero.
  const bool tail = N > 0 && static_cast<int>(list[N - 1] >> 4) * kTile + kTile > rule.kv && rule.kv < a.Lk;

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kCopyWarp) {
      // ---------------------------------------------------------- copies
      // Lane s owns ring slot s (copies of one thread complete one after
      // another, copies of several overlap); sequence K0, V0, K1, V1, ...
      bool ok = true;
      if (lane == 0 && N > 0) {
        tma_prefetch_desc(&qmap);
        tma_prefetch_desc(&kmap);
        tma_prefetch_desc(&vmap);
      }
      if (lane >= NS && lane < NS + 2 && N > 0) {
        const int t = lane - NS;
        mbar_arrive_expect_tx(&q_full[t], SK * kSlab);
        for (int s = 0; s < SK; ++s)
          tma_load_4d(sQ + (t * SK + s) * kSlab, &qmap, &q_full[t], s * 64, h, i0 + t * kTile, b);
      }
      uint32_t use = 0;  // fills of this lane's slot so far
      if (lane < NS) {
        for (int q = lane; ok && q < 2 * N; q += NS, ++use) {
          if (use && !mbar_wait(&kv_empty[lane], (use - 1) & 1u, wd)) {
            ok = false;
            break;
          }
          const int j0 = static_cast<int>(list[q >> 1] >> 4) * kTile;
          const bool is_v = q & 1;
          mbar_arrive_expect_tx(&kv_full[lane], (is_v ? SV : SK) * kSlab);
          for (int s = 0; s < (is_v ? SV : SK); ++s)
            tma_load_4d(sKV + lane * SH::kSlot + s * kSlab, is_v ? &vmap : &kmap, &kv_full[lane], s * 64, hk, j0, b);
        }
      }
      __syncwarp();
      if (tail) {
        const int q = 2 * N - 1, slot = q % NS;
        const bool got = mbar_wait(&kv_full[slot], (q / NS) & 1u, wd);
        if (got) {
          const int r0 = rule.kv % kTile;
          for (int s = 0; s < SV; ++s)
            for (int e = r0 * 8 + lane; e < kTile * 8; e += 32)
              *reinterpret_cast<uint4*>(sKV + slot * SH::kSlot + s * kSlab + e * 16) = make_uint4(0, 0, 0, 0);
          fence_async_shared();
        }
        __syncwarp();
        if (lane == 0 && got) mbar_arrive(v_tail);
      }
      // Every copy lands before the CTA can exit.
      if (lane < NS && use) mbar_wait_drain(&kv_full[lane], (use - 1) & 1u, 20000000ull);
      if (lane >= NS && lane < NS + 2 && N > 0) mbar_wait_drain(&q_full[lane - NS], 0, 20000000ull);
    } else if (warp == kMmaWarp) {
      // ------------------------------------------------------------- MMAs
      if (lane == 0 && N > 0) {
        const uint32_t idesc_s = idesc_bf16(kTile, kTile);
        const int dvn = (a.dv + 15) & ~15;
        const uint32_t idesc_o = idesc_bf16(kTile, dvn) | (1u << 16);  // B is MN-major
        const int ksteps = (a.dk + 15) / 16;
        const uint32_t q_addr = smem_u32(sQ), kv_addr = smem_u32(sKV);
        uint32_t done[2] = {0, 0};  // tiles whose P was consumed
        auto qk = [&](int t, int slot) {
          for (int s = 0; s < ksteps; ++s)
            mma_bf16(tmem + t * kTile, kmajor_swizzled_desc(q_addr + (t * SK + (s >> 2)) * kSlab + (s & 3) * 32, 128),
                     kmajor_swizzled_desc(kv_addr + slot * SH::kSlot + (s >> 2) * kSlab + (s & 3) * 32, 128), idesc_s, s > 0);
          mma_commit(&s_full[t]);
        };
        bool ok = mbar_wait(&kv_full[0], 0, wd);
        for (int t = 0; ok && t < 2; ++t) {
          ok = mbar_wait(&q_full[t], 0, wd);
          tc_fence_after_sync();
          if (ok && ((list[0] >> (2 * t)) & 3u)) qk(t, 0);
        }
        if (ok) mma_commit(&kv_empty[0]);
        for (int n = 0; ok && n < N; ++n) {
          const uint32_t e = list[n], en = n + 1 < N ? list[n + 1] : 0;
          const int vq = 2 * n + 1, vs = vq % NS, kq = 2 * n + 2, ks = kq % NS;
          ok = mbar_wait(&kv_full[vs], (vq / NS) & 1u, wd);
          if (ok && tail && n + 1 == N) ok = mbar_wait(v_tail, 0, wd);
          for (int t = 0; ok && t < 2; ++t) {
            if ((e >> (2 * t)) & 3u) {
              ok = mbar_wait(&p_ready[t], done[t] & 1u, wd);
              if (!ok) break;
              tc_fence_after_sync();
              for (int s = 0; s < kTile / 16; ++s)
                mma_bf16_ts(tmem + 2 * kTile + t * SV * 64, tmem + t * kTile + s * 8,
                            mnmajor_desc(kv_addr + vs * SH::kSlot + s * 2048), idesc_o, done[t] > 0 || s > 0);
              ++done[t];
            }
            if (n + 1 < N) {
              if (t == 0) {
                ok = mbar_wait(&kv_full[ks], (kq / NS) & 1u, wd);
                if (!ok) break;
                tc_fence_after_sync();
              }
              if ((en >> (2 * t)) & 3u) qk(t, ks);
            }
          }
          if (ok) {
            mma_commit(&kv_empty[vs]);
            if (n + 1 < N) mma_commit(&kv_empty[ks]);
          }
        }
        // The MMAs issued so far end before TMEM and shared memory are given back.
        mma_commit(&o_full[0]);
        mma_commit(&o_full[1]);
        if (!ok) mbar_wait_drain(&o_full[0], 0, 20000000ull);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ---------------------------------------------- softmax, one query per thread
    const int t = warp >> 2;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // this warp's 32 TMEM lanes
    const uint32_t s_col = tmem + lanes + t * kTile, o_col = tmem + lanes + 2 * kTile + t * SV * 64;
    int* my_docs = doc_buf + warp * kTile;
    const float c_scale = a.scale * kLog2e;
    const bool cap = a.softcap > 0.f, bias = a.slopes != nullptr;
    const float mult = cap || bias ? 1.f : c_scale;                     // x = mult * value kept
    const float cap_a = a.softcap * kLog2e, cap_k = cap ? 2.f * c_scale / a.softcap : 0.f;
    const float slope = bias ? a.slopes[h] * kLog2e : 0.f;
    const int at = my_row + a.q_offset;
    float m_ref = kNegInf, l = 0.f;
    uint32_t seen = 0;
    bool ok = true;
    for (int n = 0; n < N; ++n) {
      const uint32_t e = list[n];
      const uint32_t st = (e >> (2 * t)) & 3u;
      if (st == kSkip) continue;
      const int j0 = static_cast<int>(e >> 4) * kTile;
      if (st == kMasked && docs) {
        __syncwarp();
        for (int c = lane; c < kTile; c += 32) my_docs[c] = j0 + c < rule.kv ? doc_k[j0 + c] : -1;
        __syncwarp();
      }
      ok = mbar_wait(&s_full[t], seen & 1u, wd);
      ok = __all_sync(~0u, ok);
      if (!ok) break;
      tc_fence_after_sync();
      float s[kTile];
#pragma unroll
      for (int c = 0; c < kTile; c += 32) tmem_ld_x32f(s_col + c, s + c);
      tmem_wait_ld();
      if (cap) {
        // cap * tanh(s / cap) = cap - 2 cap / (1 + e^(2 s / cap)), in log2 units
#pragma unroll
        for (int c = 0; c < kTile; ++c)
          s[c] = fmaf(-2.f * cap_a, rcp_approx(1.f + exp2_approx(s[c] * cap_k)), cap_a);
      }
      if (bias) {
        const float f = static_cast<float>(at - j0), k = cap ? 1.f : c_scale;
#pragma unroll
        for (int c = 0; c < kTile; ++c) s[c] = fmaf(-slope, fabsf(f - static_cast<float>(c)), s[c] * k);
      }
      if (st == kMasked) {
        const int lim = my_hi - j0;
        if (docs) {
#pragma unroll
          for (int c = 0; c < kTile; c += 4) {
            const int4 d = *reinterpret_cast<const int4*>(my_docs + c);
            s[c] = c < lim && d.x == my_doc ? s[c] : kNegInf;
            s[c + 1] = c + 1 < lim && d.y == my_doc ? s[c + 1] : kNegInf;
            s[c + 2] = c + 2 < lim && d.z == my_doc ? s[c + 2] : kNegInf;
            s[c + 3] = c + 3 < lim && d.w == my_doc ? s[c + 3] : kNegInf;
          }
        } else {
#pragma unroll
          for (int c = 0; c < kTile; ++c) s[c] = c < lim ? s[c] : kNegInf;
        }
      }
      float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
      for (int c = 4; c < kTile; c += 4) {
        mx[0] = fmaxf(mx[0], s[c]);
        mx[1] = fmaxf(mx[1], s[c + 1]);
        mx[2] = fmaxf(mx[2], s[c + 2]);
        mx[3] = fmaxf(mx[3], s[c + 3]);
      }
      const float m_new = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * mult;
      const bool grow = m_new > m_ref + kGrowth;  // also: the first visible key (m_ref = -inf)
      if (__any_sync(~0u, grow)) {
        const float f = grow ? exp2_approx(m_ref - m_new) : 1.f;
        if (grow) m_ref = m_new;
        l *= f;
        if (seen) {
          for (int c = 0; c < SV * 64; c += 32) {
            float o[32];
            tmem_ld_x32f(o_col + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= f;
            tmem_st_x32(o_col + c, reinterpret_cast<uint32_t*>(o));
          }
        }
      }
      const float mu = m_ref == kNegInf ? 0.f : m_ref;
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < kTile; c += 64) {
        uint32_t p[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float p0 = exp2_approx(fmaf(s[c + 2 * i], mult, -mu));
          const float p1 = exp2_approx(fmaf(s[c + 2 * i + 1], mult, -mu));
          sum[2 * (i & 1)] += p0;
          sum[2 * (i & 1) + 1] += p1;
          const __nv_bfloat162 w = __floats2bfloat162_rn(p0, p1);
          p[i] = *reinterpret_cast<const uint32_t*>(&w);
        }
        tmem_st_x32(s_col + c / 2, p);
      }
      l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      tmem_wait_st();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_ready[t]);
      ++seen;
    }
    // ------------------------------------------------------------ output
    if (ok && seen) ok = __all_sync(~0u, mbar_wait(&o_full[t], 0, wd));
    if (ok) {
      tc_fence_after_sync();
      const float inv = l == 0.f ? 0.f : 1.f / l;
      float probe = inv * 0.f;
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.o) + b * a.os_b + static_cast<long long>(my_row) * a.os_l + h * a.os_h;
      for (int c = 0; c < a.dv; c += 32) {
        float v[32];
        if (seen) {
          tmem_ld_x32f(o_col + c, v);
          tmem_wait_ld();
        }
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float x = seen ? v[i + 2 * k] * inv : 0.f, y = seen ? v[i + 2 * k + 1] * inv : 0.f;
            if (c + i < a.dv) probe += x * 0.f + y * 0.f;
            const __nv_bfloat162 xy = __floats2bfloat162_rn(x, y);
            w[k] = *reinterpret_cast<const uint32_t*>(&xy);
          }
          if (my_row < a.Lq && c + i < a.dv) *reinterpret_cast<uint4*>(o + c + i) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      // Rows that met a non-finite value: again, key by key (attn_row).
      unsigned bad = __ballot_sync(~0u, my_row < a.Lq && !(probe == 0.f));
      while (bad) {
        const int r = __ffs(bad) - 1;
        bad &= bad - 1;
        attn_row<__nv_bfloat16>(a, b, h, i0 + warp * 32 + r);
      }
    }
    tc_fence_before_sync();
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

size_t list_bytes(int Lk) { return (static_cast<size_t>(Lk + kTile - 1) / kTile) * sizeof(uint32_t); }

template <int SK, int SV>
cudaError_t launch_shape(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const AttnArgs& a, cudaStream_t s) {
  const size_t smem = Shape<SK, SV>::kFixed + list_bytes(a.Lk);
  const cudaError_t e = smem_attr_once<attn_tc_kernel<SK, SV>>(smem);
  if (e != cudaSuccess) return e;
  const int tiles = (a.Lq + 2 * kTile - 1) / (2 * kTile);
  const long long ctas = static_cast<long long>(tiles) * a.B * a.Hq;
  if (ctas >= (1LL << 31)) return cudaErrorInvalidConfiguration;
  return launch_pdl(attn_tc_kernel<SK, SV>, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), smem, s, q, k, v, a, tiles);
}

}  // namespace

void attn_tc_box(int* box_d, int* box_l) { *box_d = 64, *box_l = kTile; }

cudaError_t launch_attn_tc(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const AttnArgs& a, cudaStream_t s) {
  if (a.dk <= 64) return a.dv <= 64 ? launch_shape<1, 1>(q, k, v, a, s) : launch_shape<1, 2>(q, k, v, a, s);
  return a.dv <= 64 ? launch_shape<2, 1>(q, k, v, a, s) : launch_shape<2, 2>(q, k, v, a, s);
}

}  // namespace cb
