// Attention on the tensor cores: bf16 views of whole 16-byte pieces.
//
// Persistent CTAs, one per SM. The queries of the heads that share a key head
// are cut into tiles of 128 of one head, heads fastest; an item is two
// neighbouring tiles t (two heads of a group, or 256 queries of one), which
// walk the visible key tiles of 128 with a running maximum and sum per query:
//   S_t = Q_t K^T        tcgen05.mma, both operands in shared memory (TMA, 128-byte swizzle),
//                        fp32 accumulator in 128 TMEM columns
//   P_t = 2^(x - m)      x = log2(e) * score, rounded to bf16 and stored over S_t
//   O_t += P_t V         tcgen05.mma with A = P_t from TMEM and B = V as it lies (rows of keys:
//                        the MN-major operand), O_t in up to 128 further columns
// Per pair of 128 x 128 tiles and 128 dims the MMAs take 2048 cycles of an SM
// and the softmax about 900 issue slots of each scheduler; what decides is the
// chain S -> P -> next S of one tile. So the two tiles take turns (the tensor
// cores work on one while the other's weights are computed), a thread holds a
// query's 128 scores in packed fp32 pairs, and nothing waits between items:
// copies run ahead through a ring that items share, a scheduler warp lists the
// next item's key tiles, and the first MMAs of an item run under the output of
// the one before.
//
// Each tile has its own MMA warp, which issues PV_t(n), then QK_t(n+1): S_t is
// overwritten only by an MMA issued after the one that reads P_t, and the
// commit after QK_t(n+1) also covers PV_t(n), so once the softmax warps see
// S_t(n+1) they may rescale O_t without another barrier. (One warp for both
// tiles was late by 2000 of 4000 cycles per pair: every wait, commit and list
// read of one tile delayed the other's MMAs.)
//
// Weights are relative to m_ref, the maximum of a query's first visible tile,
// and stay so until a tile's weights sum to more than 2^64: fp32 sums and bf16
// weights keep their relative precision at any such scale, so the running
// maximum is needed only against overflow, and an ordinary tile's maximum is
// never taken. The first tile, masked ones and those that overflow take the
// slow path: scores, mask, maximum, and l and O brought to the new one. P is
// rounded to bf16 for the second product (each weight to nearest, independent
// from key to key); l sums the unrounded weights.
//
// 4096 tokens, 16 heads on 4 key heads of 128: 102 us, 1350 TFLOP/s (0.70 of
// the measured bf16 rate); capped 137, biased 115, causal 54; 16 heads of 64:
// 86. The rest is latency: a tile's scores wait for its own weights' product,
// and two warps per scheduler do not cover all of it. Measured and not kept: P in
// columns of its own for narrow values, so that the next scores start earlier
// (86 -> 90); one path for full and masked tiles (104 -> 109).
//
// Key tiles no query of the item sees are never loaded: the list of the tiles
// to visit holds each query tile's state (skip, full, masked), nearest keys
// first: a bias by distance then has its largest scores in the first tile.
#include <cmath>
#include <type_traits>

#include "attention_common.cuh"
#include "launch_util.h"
#include "ptx.cuh"

namespace cb {

namespace {

constexpr int kTile = 128;          // queries per tile, keys per tile
constexpr int kSlab = 128 * 128;    // bytes of 128 rows x 64 bf16
constexpr int kSoftmaxWarps = 8;    // two warpgroups, one per tile
constexpr int kCopyWarp = 8, kMmaWarp = 9, kListWarp = 11;  // MMA warps 9 and 10: tiles 0 and 1
// At launch every thread holds 168 registers (the most for 12 warps); the last
// warpgroup hands some of its own to the softmax threads, which keep 128
// scores each: 256 * 224 + 128 * 56 = 384 * 168.
constexpr int kThreads = 384;
constexpr int kSoftmaxRegs = 224, kOtherRegs = 56;
static_assert(256 * kSoftmaxRegs + 128 * kOtherRegs <= kThreads * 168, "registers of the launch");
constexpr float kGrowth = 64.f;     // log2 of the largest weight sum of a tile before its maximum is taken anew
constexpr int kListReaders = kSoftmaxWarps + 3;

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
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// These are .sync.aligned: the warp is converged explicitly before each group of
// them (a lane back from a branch of its own is not otherwise sure to have rejoined).
__device__ __forceinline__ void tmem_wait_ld() {
  __syncwarp();
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void st_global_x8(void* p, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]),
               "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

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

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Capped scores: cap tanh(y), y = s / cap, as s Q(s^2) with coefficients for
// |y| <= 0.8, |error of tanh| <= 6.1e-6 (a minimax fit of degree 3 in y^2):
// packed operations on the FMA pipe, where 1 - 2 / (1 + e^(2 y)) takes two of
// the exponential unit's, which has none to spare. Scores rarely come near
// their cap; a warp that holds one that does takes the exact form for its tile.
// That form's error is a few 2^-24 of the cap: up to a cap of 1024 a few 1e-4,
// less than the weights' rounding to bf16. Larger caps are kernels of their own
// (kFarCapped), which take it only for the scores that need it; for all caps
// that would cost 510 us for 310 (4096 tokens, 16 heads of 128, cap 15).
enum { kUncapped, kCapped, kFarCapped };
constexpr float kFarCap = 1024.f;
constexpr float kTanhRange = 0.8f;
constexpr float kTanh[4] = {0.9999305605888367f, -0.3318033516407013f, 0.1240561306476593f, -0.03185783699154854f};

enum : uint32_t { kSkip = 0, kFull = 1, kMasked = 2 };

struct Item {
  int b, hk;
  int h[2], i0[2];  // per tile; a tile past the last one starts at Lq: it has no query
};
// What the scheduler warp says about an item.
struct ItemInfo {
  Item it;     // worked out once: the divisions took a softmax thread about 1000 cycles per item
  int n;       // tiles in the list
  int kv;      // keys of the sequence
  int prefix;
  int tail;    // 1: the tile of key kv, if listed, holds rows past it, whose values must become zero
  float slope[2];  // log2(e) times the slopes of the two tiles' heads
};

// Least and greatest document of key tiles [n0, n0 + count) of sequence b, into
// cache[0 .. count), by `warps` warps.  A key past the end counts as padding.
constexpr int kDocTiles = 512;  // tiles whose ranges are kept: 65536 keys
__device__ __forceinline__ void scan_docs(const AttnArgs& a, int b, int kv, int2* cache, int n0, int count, int warp, int warps) {
  constexpr int kBatch = 4;  // tiles whose ids are in flight together
  const int lane = threadIdx.x & 31;
  const int* doc_k = a.doc_k + static_cast<long long>(b) * a.Lk;
  const bool vec = a.Lk % 4 == 0 && (reinterpret_cast<uintptr_t>(a.doc_k) & 15) == 0;
  for (int x0 = warp * kBatch; x0 < count; x0 += warps * kBatch) {
    int lo[kBatch], hi[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int j0 = (n0 + x0 + u) * kTile;
      int4 d = make_int4(-1, -1, -1, -1);
      if (vec && j0 + kTile <= kv) {
        d = __ldg(reinterpret_cast<const int4*>(doc_k + j0) + lane);
      } else {
        if (j0 + lane < kv) d.x = __ldg(doc_k + j0 + lane);
        if (j0 + lane + 32 < kv) d.y = __ldg(doc_k + j0 + lane + 32);
        if (j0 + lane + 64 < kv) d.z = __ldg(doc_k + j0 + lane + 64);
        if (j0 + lane + 96 < kv) d.w = __ldg(doc_k + j0 + lane + 96);
      }
      lo[u] = min(min(d.x, d.y), min(d.z, d.w));
      hi[u] = max(max(d.x, d.y), max(d.z, d.w));
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int2 r = make_int2(__reduce_min_sync(~0u, lo[u]), __reduce_max_sync(~0u, hi[u]));
      if (lane == u && x0 + u < count) cache[x0 + u] = r;
    }
  }
  __syncwarp();
}

template <int SK, int SV>
struct Shape {
  static constexpr int kSlot = (SK > SV ? SK : SV) * kSlab;  // one ring slot: a K or a V tile
  static constexpr int kStages = SK == 2 || SV == 2 ? 4 : 8;
  static constexpr int kQ = 2 * SK * kSlab;
  static constexpr int kFixed = kQ + kStages * kSlot + 4 * kTile * 4 /* queries' documents */ + 1024 /* barriers, item infos */ + 1024 /* alignment */;
};

// Work items of the launch, longest first (under a causal mask the last query
// tiles).  CTA c takes items c, 2 g - 1 - c, 2 g + c, ... of g CTAs: turning
// round after each row evens long and short ones out.
__device__ __forceinline__ int item_of(int k) {
  return k * gridDim.x + (k & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}
__device__ __forceinline__ Item item_at(const AttnArgs& a, int pairs, int item) {
  const int seqs = a.B * (a.Hq / a.group), bh = item % seqs, u = 2 * (pairs - 1 - item / seqs);
  Item it;
  it.b = bh / (a.Hq / a.group);
  it.hk = bh % (a.Hq / a.group);
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int q = (u + t) / a.group;
    it.h[t] = it.hk * a.group + (u + t) % a.group;
    it.i0[t] = min(q * kTile, a.Lq);
  }
  return it;
}

// CAP, BIAS: how scores are capped, whether they are biased (a branch per tile would make
// every path keep the 128 scores in the same registers).
template <int SK, int SV, int CAP, bool BIAS>
__global__ void __launch_bounds__(kThreads, 1)
attn_tc_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
               const __grid_constant__ CUtensorMap vmap, const __grid_constant__ AttnArgs a, int pairs, int items, int list_len) {
  using SH = Shape<SK, SV>;
  constexpr int NS = SH::kStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sKV = smem + SH::kQ;
  int* q_docs = reinterpret_cast<int*>(sKV + NS * SH::kSlot);  // [2 lists][2 tiles][128]: documents of the queries
  uint64_t* q_full = reinterpret_cast<uint64_t*>(q_docs + 4 * kTile);
  uint64_t* q_empty = q_full + 2;
  uint64_t* kv_full = q_empty + 2;
  uint64_t* kv_empty = kv_full + NS;
  uint64_t* s_full = kv_empty + NS;
  uint64_t* p_ready = s_full + 2;
  uint64_t* o_full = p_ready + 2;
  uint64_t* o_free = o_full + 2;
  uint64_t* list_full = o_free + 2;
  uint64_t* list_free = list_full + 2;
  uint64_t* drain = list_free + 2;  // all MMAs of a tile's warp are over
  uint64_t* v_tail = drain + 2;  // the values past the end of a tail tile are zero
  int* turn = reinterpret_cast<int*>(v_tail + 1);  // 1 while an MMA warp issues a tile's MMAs
  ItemInfo* info = reinterpret_cast<ItemInfo*>(v_tail + 2);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(info + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* lists = reinterpret_cast<uint32_t*>(reinterpret_cast<uint8_t*>(q_full) + 1024);  // [2][list_len]
  int2* doc_cache = reinterpret_cast<int2*>(lists + 2 * ((list_len + 1) & ~1));            // [2][kDocTiles] with documents

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(&q_full[t], 1);
      mbar_init(&q_empty[t], 1);
      mbar_init(&s_full[t], 1);
      mbar_init(&p_ready[t], 4);
      mbar_init(&o_full[t], 1);
      mbar_init(&o_free[t], 4);
      mbar_init(&list_full[t], 1);
      mbar_init(&drain[t], 1);
      mbar_init(&list_free[t], kListReaders);
    }
    for (int s = 0; s < NS; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 2);
    }
    mbar_init(v_tail, 2);
    *abort_flag = 0;
    *turn = 0;
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
  const int rounds = (items + gridDim.x - 1) / gridDim.x;
  // The first two items' document ranges by every warp: nothing hides their latency yet.
  const int key_tiles = (a.Lk + kTile - 1) / kTile;
  if (a.doc_k && key_tiles <= kDocTiles) {
    for (int k = 0; k < 2; ++k)
      if (k < rounds && item_of(k) < items) {
        const int b = item_at(a, pairs, item_of(k)).b;
        scan_docs(a, b, seq_rule(a, b).kv, doc_cache + k * kDocTiles, 0, key_tiles, warp, kThreads / 32);
      }
    __syncthreads();
  }

  if (warp >= kSoftmaxWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kListWarp) {
      // ------------------------------------------------------------ lists
      bool ok = true;
      int cached0 = rounds > 0 && item_of(0) < items ? item_at(a, pairs, item_of(0)).b : -1;  // whose ranges the caches hold
      int cached1 = rounds > 1 && item_of(1) < items ? item_at(a, pairs, item_of(1)).b : -1;
      for (int k = 0, item; ok && k < rounds; ++k) {
        if ((item = item_of(k)) >= items) break;
        const int buf = k & 1;
        if (k >= 2) ok = mbar_wait(&list_free[buf], ((k >> 1) - 1) & 1u, wd);
        ok = __all_sync(~0u, ok);
        if (!ok) break;
        const Item it = item_at(a, pairs, item);
        const SeqRule rule = seq_rule(a, it.b);
        uint32_t* list = lists + buf * list_len;
        int hi_lo[2], hi_hi[2];  // per query tile: keys that all / some of its queries see, before documents
        for (int t = 0; t < 2; ++t) {
          const int r0 = it.i0[t], r1 = min(a.Lq, r0 + kTile) - 1;
          hi_lo[t] = r0 <= r1 ? row_end(a, rule, r0) : 0;
          hi_hi[t] = r0 <= r1 ? row_end(a, rule, r1) : 0;
        }
        const int all = (max(hi_hi[0], hi_hi[1]) + kTile - 1) / kTile;
        int kept = 0;
        if (!a.doc_k) {
          // from the tile of the item's last query down to the first, then the ones past it
          const int near = min(all, max(0, (min(a.Lq, max(it.i0[0] + (it.i0[0] < a.Lq) * kTile, it.i0[1] < a.Lq ? it.i0[1] + kTile : 0)) - 1 + a.q_offset) / kTile + 1));
          for (int x = lane; x < all; x += 32) {
            const int n = x < near ? near - 1 - x : x;
            uint32_t e = n << 4;
            for (int t = 0; t < 2; ++t)
              e |= (n * kTile >= hi_hi[t] ? kSkip : (n + 1) * kTile <= hi_lo[t] ? kFull : kMasked) << (2 * t);
            list[x] = e;
          }
          kept = all;
        } else {
          int dlo[2], dhi[2];  // documents of each tile's queries; hi_lo = 0 where one is padding
          for (int t = 0; t < 2; ++t) {
            int lo = 0x7fffffff, hi = -1, pad = 0;
            for (int c = lane; c < kTile; c += 32) {
              const int i = it.i0[t] + c;
              const int d = i < a.Lq ? a.doc_q[static_cast<long long>(it.b) * a.Lq + i] : -1;
              q_docs[(buf * 2 + t) * kTile + c] = d;
              if (d >= 0) lo = min(lo, d), hi = max(hi, d);
              pad |= i < a.Lq && d < 0;
            }
            dlo[t] = __reduce_min_sync(~0u, lo);
            dhi[t] = __reduce_max_sync(~0u, hi);
            if (__any_sync(~0u, pad)) hi_lo[t] = 0;
          }
          // from the last tile down; ranges of up to kDocTiles tiles at a time
          for (int end = all; end > 0; end -= kDocTiles) {
            const int n0 = key_tiles <= kDocTiles ? 0 : max(0, end - kDocTiles);
            int2* cache = doc_cache + buf * kDocTiles;
            if (key_tiles > kDocTiles) scan_docs(a, it.b, rule.kv, cache, n0, end - n0, 0, 1);
            else if (k >= 2 && it.b != (buf ? cached1 : cached0)) scan_docs(a, it.b, rule.kv, cache, 0, key_tiles, 0, 1);
            for (int x0 = end - 1; x0 >= n0; x0 -= 32) {
              const int n = x0 - lane;
              uint32_t e = 0;
              if (n >= n0) {
                const int l = cache[n - n0].x, h = cache[n - n0].y;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                  uint32_t st = n * kTile >= hi_hi[t] || h < dlo[t] || l > dhi[t] ? kSkip : kMasked;
                  if (st == kMasked && l == h && dlo[t] == dhi[t] && l == dlo[t] && (n + 1) * kTile <= hi_lo[t]) st = kFull;
                  e |= st << (2 * t);
                }
              }
              const unsigned keep = __ballot_sync(~0u, e != 0);
              if (e) list[kept + __popc(keep & ((1u << lane) - 1))] = e | (n << 4);
              kept += __popc(keep);
            }
          }
          (buf ? cached1 : cached0) = it.b;
        }
        __syncwarp();
        if (lane == 0) {
          info[buf] = {it, kept, rule.kv, rule.prefix, rule.kv < a.Lk && rule.kv % kTile != 0,
                       {a.slopes ? a.slopes[it.h[0]] * kLog2e : 0.f, a.slopes ? a.slopes[it.h[1]] * kLog2e : 0.f}};
          mbar_arrive(&list_full[buf]);
        }
      }
    } else if (warp == kCopyWarp) {
      // ----------------------------------------------------------- copies
      // Lane s owns ring slot s (copies of one thread complete one after
      // another, copies of several overlap) of the sequence K0, V0, K1, V1,
      // ... that runs on from item to item; two further lanes own Q_0, Q_1.
      if (lane == 0) {
        tma_prefetch_desc(&qmap);
        tma_prefetch_desc(&kmap);
        tma_prefetch_desc(&vmap);
      }
      bool ok = true;
      uint32_t use = 0;  // fills of this lane's slot or Q tile so far
      long long base = 0;
      for (int k = 0; ok && k < rounds; ++k) {
        if (item_of(k) >= items) break;
        const int buf = k & 1;
        ok = mbar_wait(&list_full[buf], (k >> 1) & 1u, wd);
        ok = __all_sync(~0u, ok);
        if (!ok) break;
        const int n = info[buf].n;
        const Item it = info[buf].it;
        const uint32_t* list = lists + buf * list_len;
        if (n > 0 && lane >= NS && lane < NS + 2) {
          const int t = lane - NS;
          ok = use == 0 || mbar_wait(&q_empty[t], (use - 1) & 1u, wd);
          if (ok) {
            mbar_arrive_expect_tx(&q_full[t], SK * kSlab);
            for (int s = 0; s < SK; ++s)
              tma_load_4d(sQ + (t * SK + s) * kSlab, &qmap, &q_full[t], s * 64, it.h[t], it.i0[t], it.b);
            ++use;
          }
        }
        if (lane < NS) {
          // this lane's first place in the item: base + q == lane mod NS
          for (int q = (lane - static_cast<int>(base % NS) + NS) % NS; q < 2 * n; q += NS) {
            ok = use == 0 || mbar_wait(&kv_empty[lane], (use - 1) & 1u, wd);
            if (!ok) break;
            const int j0 = static_cast<int>(list[q >> 1] >> 4) * kTile;
            const bool is_v = q & 1;
            mbar_arrive_expect_tx(&kv_full[lane], (is_v ? SV : SK) * kSlab);
            for (int s = 0; s < (is_v ? SV : SK); ++s)
              tma_load_4d(sKV + lane * SH::kSlot + s * kSlab, is_v ? &vmap : &kmap, &kv_full[lane], s * 64, it.hk, j0, it.b);
            ++use;
          }
        }
        base += 2 * n;
        ok = __all_sync(~0u, ok);
        if (lane == 0) mbar_arrive(&list_free[buf]);
      }
      // Every copy lands before the CTA can exit.
      if (use && lane < NS) mbar_wait_drain(&kv_full[lane], (use - 1) & 1u, 20000000ull);
      if (use && lane >= NS && lane < NS + 2) mbar_wait_drain(&q_full[lane - NS], (use - 1) & 1u, 20000000ull);
    } else {
      // ------------------------------------------------------------- MMAs
      // The whole warp walks the steps together and one elected lane issues,
      // so that descriptors stay in uniform registers.  They advance by
      // 16-byte units in their low word; the high word is a constant.
      // (Built anew by a lone lane, each took longer than its MMA: 75 to 150
      // cycles against 64.)
      const int t = warp - kMmaWarp;
      const uint32_t idesc_s = idesc_bf16(kTile, kTile);
      const uint32_t idesc_o = idesc_bf16(kTile, (a.dv + 15) & ~15) | (1u << 16);  // B is MN-major
      const uint32_t q_lo = static_cast<uint32_t>(kmajor_swizzled_desc(smem_u32(sQ), 128)) + t * (SK * kSlab >> 4);
      const uint32_t k_lo = static_cast<uint32_t>(kmajor_swizzled_desc(smem_u32(sKV), 128));
      const uint32_t v_lo = static_cast<uint32_t>(mnmajor_desc(smem_u32(sKV)));
      constexpr uint64_t kHi = (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
      const uint32_t s_tmem = tmem + t * kTile, o_tmem = tmem + 2 * kTile + t * SV * 64;
      const bool leader = elect_one();
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        ok = __all_sync(~0u, ok && mbar_wait(bar, parity & 1u, wd));
        return ok;
      };
      // The tensor pipe for one tile's PV and QK at a time: interleaved with the
      // other tile's they would take twice as long each, and the two tiles'
      // softmax would then run side by side instead of under those MMAs.
      auto take = [&] {
        if (leader) {
          const uint64_t t0 = global_timer_ns();
          for (int spins = 1; atomicCAS_block(turn, 0, 1) != 0; ++spins)
            if ((spins & 63) == 0 && (*abort_flag || global_timer_ns() - t0 > a.timeout_ns)) break;
        }
        __syncwarp();
      };
      auto give = [&] {
        if (leader) atomicExch_block(turn, 0);
        __syncwarp();
      };
      // One key tile of one item; `seq`: its K's place in the ring's sequence.
      struct Step {
        uint32_t state, seq;
        bool last;
        int tail;  // rows of a tail tile that are keys, else 0
      };
      int k = -1, n = 0, count = 0, tail_tile = -1, tail_rows = 0;
      uint32_t seq = 0;
      // Parities of the next waits (Q and o_free: of the phase before the next one), and two facts about the item at
      // hand: its Q was waited for, its O was begun.
      enum : uint32_t { kP = 1, kTail = 2, kQ = 4, kO = 8, kHaveQ = 16, kBegun = 32 };
      uint32_t bits = kQ | kO;
      // kNone: no further step (or a wait gave up). ahead: the last step's second product is still to be issued, and
      // kLater says that the item after its own is empty. Past two such items the next list would come only when the
      // softmax warps have left the first, and so the output that waits for that product.
      enum Fetched { kNone, kStep, kLater };
      auto fetch = [&](Step* s, bool ahead) {
        while (n == count) {
          ++k;
          if (k >= rounds || item_of(k) >= items) return kNone;
          if (!wait(&list_full[k & 1], k >> 1)) return kNone;
          n = 0;
          count = __shfl_sync(~0u, info[k & 1].n, 0);
          const int kv = __shfl_sync(~0u, info[k & 1].kv, 0);
          tail_tile = __shfl_sync(~0u, info[k & 1].tail, 0) ? kv / kTile : -1;
          tail_rows = kv % kTile;
          if (count == 0) {
            if (leader) mbar_arrive(&list_free[k & 1]);
            if (ahead) return kLater;
          }
        }
        const uint32_t e = __shfl_sync(~0u, lists[(k & 1) * list_len + n], 0);
        s->state = (e >> (2 * t)) & 3u;
        s->seq = seq;
        if (n == 0) bits = (bits ^ kQ) & ~kHaveQ;
        s->last = ++n == count;
        s->tail = static_cast<int>(e >> 4) == tail_tile ? tail_rows : 0;
        seq += 2;
        if (s->last && leader) mbar_arrive(&list_free[k & 1]);
        return kStep;
      };
      auto k_wait = [&](const Step& s) {
        wait(&kv_full[s.seq % NS], s.seq / NS);
        // Q_t has landed before its buffer is given back, also where no key tile of the item used it: a second
        // load into a barrier whose first is still under way would be one arrival too many.
        if ((s.state || s.last) && !(bits & kHaveQ)) {
          bits |= kHaveQ;
          wait(&q_full[t], (bits & kQ) != 0);
        }
      };
      auto qk = [&](const Step& s) {
        tc_fence_after_sync();
        const uint32_t kl = k_lo + s.seq % NS * (SH::kSlot >> 4);
        if (leader) {
          if (s.state) {
#pragma unroll
            for (int x = 0; x < 4 * SK; ++x) {  // dims past dk are zero in both operands
              const uint32_t off = ((x >> 2) * kSlab + (x & 3) * 32) >> 4;
              mma_bf16(s_tmem, kHi | (q_lo + off), kHi | (kl + off), idesc_s, x > 0);
            }
            mma_commit(&s_full[t]);
          }
          mma_commit(&kv_empty[s.seq % NS]);
          if (s.last) mma_commit(&q_empty[t]);
        }
        __syncwarp();
      };
      Step cur, nxt;
      bool held = false;  // cur is a step whose second product is still to be issued
      for (;;) {
        const Fetched next = fetch(&nxt, held);
        const bool more = next == kStep;
        if (!ok || !(held || more)) break;
        const uint32_t vq = held ? cur.seq + 1 : 0, vs = vq % NS, vl = v_lo + vs * (SH::kSlot >> 4);
        if (held) wait(&kv_full[vs], vq / NS);
        if (ok && held && cur.tail) {  // values past the sequence's end, whatever they are, become zero
          if (t == 0) {
            for (int s = 0; s < SV; ++s)
              for (int e = cur.tail * 8 + lane; e < kTile * 8; e += 32)
                *reinterpret_cast<uint4*>(sKV + vs * SH::kSlot + s * kSlab + e * 16) = make_uint4(0, 0, 0, 0);
            fence_async_shared();
            __syncwarp();
          }
          if (lane == 0) mbar_arrive(v_tail);  // both warps: neither is ever two tails ahead of the other
          wait(v_tail, (bits & kTail) != 0);
          bits ^= kTail;
        }
        if (ok && more) k_wait(nxt);
        if (!ok) break;
        if (held && cur.state) {
          const uint32_t begun = (bits & kBegun) != 0;
          if (!begun) wait(&o_free[t], (bits & kO) != 0);  // at once before the first item's
          if (!ok || !wait(&p_ready[t], bits & kP)) break;
          take();
          tc_fence_after_sync();
          if (leader) {
#pragma unroll
            for (int x = 0; x < kTile / 16; ++x)
              mma_bf16_ts(o_tmem, s_tmem + x * 8, kHi | (vl + x * (2048 >> 4)), idesc_o, x > 0 ? 1u : begun);
          }
          __syncwarp();
          bits = (bits ^ kP) | kBegun;
        }
        if (held && cur.last && (bits & kBegun)) {
          if (leader) mma_commit(&o_full[t]);
          __syncwarp();
          bits = (bits ^ kO) & ~kBegun;
        }
        if (more) qk(nxt);
        if (held) {
          if (cur.state) give();
          if (leader) mma_commit(&kv_empty[vs]);
          __syncwarp();
        }
        held = more;
        cur = nxt;
      }
      __syncwarp();
      if (leader) {  // the MMAs and arrivals issued so far end before TMEM and shared memory are given back
        mma_commit(&drain[t]);
        mbar_wait_drain(&drain[t], 0, 20000000ull);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ---------------------------------------- softmax, one query per thread
    const int t = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // this warp's 32 TMEM lanes
    const uint32_t s_col = tmem + lanes + t * kTile, o_col = tmem + lanes + 2 * kTile + t * SV * 64;
    // 32-byte stores of the output, where its rows allow them: a store instruction touches 32 rows, and costs
    // by the row
    const bool wide = ((reinterpret_cast<uintptr_t>(a.o) | (a.os_b * 2) | (a.os_l * 2) | (a.os_h * 2)) & 31) == 0 && a.dv % 16 == 0;
    uint32_t s_seen = 0, o_seen = 0;
    bool ok = true;
    // What a thread needs of an item. The next one's is read before an item's output: the wait for the last
    // product covers it.
    struct Mine {
      int b, i0, h, n, kv, doc, hi;
      float slope;
    } me, next;
    auto read = [&](int k, Mine* m) {  // false: no such item, or a wait gave up (ok)
      if (k >= rounds || item_of(k) >= items) return false;
      const int buf = k & 1;
      ok = __all_sync(~0u, mbar_wait(&list_full[buf], (k >> 1) & 1u, wd));
      if (!ok) return false;
      const ItemInfo inf = info[buf];
      m->b = inf.it.b, m->i0 = t ? inf.it.i0[1] : inf.it.i0[0], m->h = t ? inf.it.h[1] : inf.it.h[0];
      m->n = inf.n, m->kv = inf.kv, m->slope = t ? inf.slope[1] : inf.slope[0];
      m->doc = a.doc_q ? q_docs[(buf * 2 + t) * kTile + row] : 0;
      // a row that sees nothing (hi 0) is dead: whatever it computes is dropped
      m->hi = m->i0 + row < a.Lq && m->doc >= 0 ? row_end(a, SeqRule{inf.kv, inf.prefix}, m->i0 + row) : 0;
      return true;
    };
    bool more = read(0, &me);
    for (int k = 0; more; ++k, me = next) {
      const int buf = k & 1, b = me.b, i0 = me.i0, h = me.h, i = i0 + row, doc = me.doc, hi = me.hi, at = i + a.q_offset;
      const uint32_t* list = lists + buf * list_len;
      const float slope = me.slope;
      float m_ref = kNegInf, l = 0.f;
      bool any = false;
      for (int n = 0; n < me.n; ++n) {
        const uint32_t e = list[n], st = (e >> (2 * t)) & 3u;
        if (st == kSkip) continue;
        const int j0 = static_cast<int>(e >> 4) * kTile;
        // Bit c of seen: this row sees key j0 + c. Found before the scores are waited for.
        uint32_t seen[4] = {~0u, ~0u, ~0u, ~0u};
        if (st == kMasked) {
          if (a.doc_k) {
            int key_doc[4];  // documents of keys lane + 32 x
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int j = j0 + lane + 32 * x;
              key_doc[x] = j < me.kv ? a.doc_k[static_cast<long long>(b) * a.Lk + j] : -1;
            }
            // The documents of a warp's rows are few: one round each.
            unsigned rows = ~0u;
            while (rows) {
              const int d = __shfl_sync(~0u, doc, __ffs(rows) - 1);
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const uint32_t same = __ballot_sync(~0u, key_doc[x] == d);
                if (doc == d) seen[x] = same;
              }
              rows &= ~__ballot_sync(~0u, doc == d);
            }
          }
          const int lim = hi - j0;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int n_seen = min(max(lim - 32 * x, 0), 32);
            seen[x] &= n_seen == 32 ? ~0u : (1u << n_seen) - 1;
          }
        }
        ok = __all_sync(~0u, mbar_wait(&s_full[t], s_seen & 1u, wd));
        if (!ok) break;
        ++s_seen;
        tc_fence_after_sync();
        float s[kTile];
        __syncwarp();
#pragma unroll
        for (int c = 0; c < kTile; c += 32) tmem_ld_x32f(s_col + c, s + c);
        tmem_wait_ld();
        f2 sum[2];
        // Thirty-two weights at a time, two per call of `pair`, into TMEM.
        auto store_weights = [&](auto pair) {
          sum[0] = sum[1] = 0;
          __syncwarp();
#pragma unroll
          for (int c = 0; c < kTile; c += 32) {
            uint32_t p[16];
#pragma unroll
            for (int u = 0; u < 16; ++u) {
              float p0, p1;
              unpack2(pair(c + 2 * u), p0, p1);
              p0 = exp2_approx(p0);
              p1 = exp2_approx(p1);
              sum[u & 1] = add2(sum[u & 1], pack2(p0, p1));
              const __nv_bfloat162 w = __floats2bfloat162_rn(p0, p1);
              p[u] = *reinterpret_cast<const uint32_t*>(&w);
            }
            tmem_st_x16(s_col + c / 2, p);
          }
        };
        auto total = [&] {
          float s0, s1;
          unpack2(add2(sum[0], sum[1]), s0, s1);
          return s0 + s1;
        };
        // ------------------------------------------------ an ordinary tile
        bool fast = st == kFull && !__any_sync(~0u, hi > 0 && m_ref == kNegInf);
        // -slope |at - j| = +-slope (j - at) where a row's visible keys lie on one side of it: side * slope * (j - at)
        const float f_at = static_cast<float>(at - j0);
        float side = 0.f;
        if constexpr (BIAS) {
          if (__all_sync(~0u, min(hi, j0 + kTile) - 1 <= at || hi == 0)) side = slope;
          else if (__all_sync(~0u, at <= j0 || hi == 0)) side = -slope;
          fast = fast && side != 0.f;
        }
        // The bias of keys c, c + 1 plus `more`, for c a multiple of 32; each next pair of keys adds 2 * side.
        auto bias_at = [&](int c, float more) {
          const float y = fmaf(side, static_cast<float>(c) - f_at, more);
          return pack2(y, y + side);
        };
        const f2 bias_step = pack2(2.f * side, 2.f * side);
        bool in_range = true;
        if constexpr (CAP != kUncapped) {
          float big[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < kTile; c += 8)
#pragma unroll
            for (int u = 0; u < 4; ++u) big[u] = max3(big[u], fabsf(s[c + 2 * u]), fabsf(s[c + 2 * u + 1]));
          in_range = __all_sync(~0u, max3(fmaxf(big[0], big[1]), big[2], big[3]) * a.tc.reach <= kTanhRange);
          fast = fast && in_range;
        }
        auto cap_gain = [&](f2 x) {  // Q(x^2) with the cap's scales: x times it is log2(e) cap tanh(x / cap)
          const f2 z = mul2(x, x);
          f2 g = fma2(z, pack2(a.tc.poly[3], a.tc.poly[3]), pack2(a.tc.poly[2], a.tc.poly[2]));
          g = fma2(z, g, pack2(a.tc.poly[1], a.tc.poly[1]));
          return fma2(z, g, pack2(a.tc.poly[0], a.tc.poly[0]));
        };
        float tile_sum = 0.f;
        f2 y2 = 0;
        if (fast) {
          const float mu = -m_ref;
          const f2 mu2 = pack2(mu, mu);
          store_weights([&](int c) {
            const f2 x = pack2(s[c], s[c + 1]);
            f2 g;
            if constexpr (CAP != kUncapped) g = cap_gain(x);
            else g = pack2(a.tc.gain, a.tc.gain);
            if constexpr (BIAS) {
              y2 = c % 32 == 0 ? bias_at(c, mu) : add2(y2, bias_step);
              return fma2(x, g, y2);
            } else {
              return fma2(x, g, mu2);
            }
          });
          tile_sum = total();
          fast = !__any_sync(~0u, hi > 0 && !(tile_sum <= 0x1p64f));
        }
        if (!fast) {
          tmem_wait_st();  // weights of an attempt that overflowed
          // ------------------------- scores, mask, maximum; then the weights
          // x = mult * s from here on
          float mult = a.tc.gain;
          if constexpr (CAP != kUncapped) {
            if (in_range) {
#pragma unroll
              for (int c = 0; c < kTile; c += 2) {
                const f2 x = pack2(s[c], s[c + 1]);
                unpack2(mul2(x, cap_gain(x)), s[c], s[c + 1]);
              }
            } else if constexpr (CAP == kCapped) {
#pragma unroll
              for (int c = 0; c < kTile; ++c)
                s[c] = fmaf(-2.f * a.tc.cap_out, rcp_approx(1.f + exp2_approx(s[c] * (2.f * kLog2e * a.tc.cap_in))), a.tc.cap_out);
            } else {
#pragma unroll
              for (int c = 0; c < kTile; c += 2) {
                const f2 x = pack2(s[c], s[c + 1]);
                float y[2];
                unpack2(mul2(x, cap_gain(x)), y[0], y[1]);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const float d = fabsf(s[c + e]);
                  const float far = fmaf(-2.f * a.tc.cap_out, rcp_approx(1.f + exp2_approx(d * (2.f * kLog2e * a.tc.cap_in))), a.tc.cap_out);
                  s[c + e] = d * a.tc.reach <= kTanhRange ? y[e] : copysignf(far, s[c + e]);
                }
              }
            }
            mult = 1.f;
          }
          if constexpr (BIAS) {
            if (side != 0.f) {
              const f2 g2 = pack2(mult, mult);
#pragma unroll
              for (int c = 0; c < kTile; c += 2) {
                y2 = c % 32 == 0 ? bias_at(c, 0.f) : add2(y2, bias_step);
                unpack2(fma2(pack2(s[c], s[c + 1]), g2, y2), s[c], s[c + 1]);
              }
            } else {
#pragma unroll
              for (int c = 0; c < kTile; ++c) s[c] = fmaf(-slope, fabsf(f_at - static_cast<float>(c)), s[c] * mult);
            }
            mult = 1.f;
          }
          if (st == kMasked) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              if (!__all_sync(~0u, seen[x] == ~0u)) {
#pragma unroll
                for (int c = 0; c < 32; ++c) s[32 * x + c] = (seen[x] >> c) & 1 ? s[32 * x + c] : kNegInf;
              }
            }
          }
          float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int c = 4; c + 8 <= kTile; c += 8)
#pragma unroll
            for (int u = 0; u < 4; ++u) mx[u] = max3(mx[u], s[c + 2 * u], s[c + 2 * u + 1]);
          const float rest = fmaxf(max3(s[kTile - 4], s[kTile - 3], s[kTile - 2]), s[kTile - 1]);
          const float m_new = max3(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]), rest) * mult;
          const bool grow = hi > 0 && m_new > m_ref + kGrowth;  // also: the first visible key (m_ref = -inf)
          if (__any_sync(~0u, grow)) {
            const float f = grow ? exp2_approx(m_ref - m_new) : 1.f;
            if (grow) m_ref = m_new;
            l *= f;
            if (any) {
#pragma unroll 1
              for (int c = 0; c < SV * 64; c += 16) {
                uint32_t o[16];
                tmem_ld_x16(o_col + c, o);
                tmem_wait_ld();
#pragma unroll
                for (int u = 0; u < 16; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * f);
                __syncwarp();
                tmem_st_x16(o_col + c, o);
              }
            }
          }
          const float mu = m_ref == kNegInf ? 0.f : -m_ref;
          const f2 mu2 = pack2(mu, mu), mult2 = pack2(mult, mult);
          store_weights([&](int c) { return fma2(pack2(s[c], s[c + 1]), mult2, mu2); });
          tile_sum = total();
        }
        any = true;
        l += tile_sum;
        tmem_wait_st();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_ready[t]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&list_free[buf]);
      if (!ok) break;
      more = read(k + 1, &next);
      if (!ok) break;
      // ---------------------------------------------------------- output
      if (any) {
        ok = __all_sync(~0u, mbar_wait(&o_full[t], o_seen & 1u, wd));
        if (!ok) break;
        ++o_seen;
        tc_fence_after_sync();
      }
      const bool live = any && hi > 0;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const f2 inv2 = pack2(inv, inv);
      f2 probe[2] = {mul2(inv2, 0), 0};  // 0 times every value: NaN where one is not finite
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.o) + b * a.os_b + static_cast<long long>(i) * a.os_l + h * a.os_h;
#pragma unroll
      for (int d0 = 0; d0 < SV * 64; d0 += 16) {
        if (d0 >= a.dv) break;
        uint32_t v[16], w[8];
        if (any) {
          tmem_ld_x16(o_col + d0, v);
          tmem_wait_ld();
        }
        const bool second = d0 + 8 < a.dv;  // dims come in eights
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const f2 y = mul2(pack2(__uint_as_float(v[2 * u]), __uint_as_float(v[2 * u + 1])), inv2);
          if (u < 4 || second) probe[u & 1] = fma2(y, 0, probe[u & 1]);
          float y0, y1;
          unpack2(y, y0, y1);
          const __nv_bfloat162 yz = __floats2bfloat162_rn(y0, y1);
          w[u] = live ? *reinterpret_cast<const uint32_t*>(&yz) : 0u;
        }
        if (i < a.Lq) {
          if (wide) {
            st_global_x8(out + d0, w);
          } else {
            *reinterpret_cast<uint4*>(out + d0) = make_uint4(w[0], w[1], w[2], w[3]);
            if (second) *reinterpret_cast<uint4*>(out + d0 + 8) = make_uint4(w[4], w[5], w[6], w[7]);
          }
        }
      }
      float probe0, probe1;
      unpack2(add2(probe[0], probe[1]), probe0, probe1);
      if (any) {
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&o_free[t]);
      }
      // Rows that met a hidden value that is not finite: again, key by key.
      unsigned bad = __ballot_sync(~0u, i < a.Lq && live && !(probe0 + probe1 == 0.f));
      if (bad) {
        const SeqRule rule = seq_rule(a, b);
        const int end = min(rule.kv, (row_end(a, rule, min(a.Lq, i0 + kTile) - 1) + kTile - 1) / kTile * kTile);
        bad = rows_to_redo<__nv_bfloat16, true>(a, b, h / a.group, end, (bad >> lane) & 1, hi, doc, l);
        for (; bad; bad &= bad - 1) attn_row<__nv_bfloat16, true>(a, b, h, i0 + (warp & 3) * 32 + __ffs(bad) - 1);
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

size_t list_len(int Lk) { return static_cast<size_t>(Lk + kTile - 1) / kTile; }

template <int SK, int SV, int CAP, bool BIAS>
cudaError_t launch_one(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const AttnArgs& a, int sms, cudaStream_t s) {
  const size_t smem = Shape<SK, SV>::kFixed + 2 * ((list_len(a.Lk) + 1) & ~size_t(1)) * sizeof(uint32_t) +
                      (a.doc_k ? 2 * kDocTiles * sizeof(int2) : 0);
  const cudaError_t e = smem_attr_once<attn_tc_kernel<SK, SV, CAP, BIAS>>(smem);
  if (e != cudaSuccess) return e;
  const long long tiles = static_cast<long long>((a.Lq + kTile - 1) / kTile) * a.group, pairs = (tiles + 1) / 2;
  const long long items = pairs * a.B * (a.Hq / a.group);
  if (items >= (1LL << 30)) return cudaErrorInvalidConfiguration;
  const int grid = static_cast<int>(items < sms ? items : sms);
  return launch_pdl(attn_tc_kernel<SK, SV, CAP, BIAS>, dim3(grid), dim3(kThreads), smem, s, q, k, v, a, static_cast<int>(pairs),
                    static_cast<int>(items), static_cast<int>(list_len(a.Lk)));
}

template <int SK, int SV>
cudaError_t launch_shape(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const AttnArgs& a, int sms, cudaStream_t s) {
  auto capped = [&](auto cap) {
    return a.slopes ? launch_one<SK, SV, cap(), true>(q, k, v, a, sms, s) : launch_one<SK, SV, cap(), false>(q, k, v, a, sms, s);
  };
  if (a.softcap > kFarCap) return capped(std::integral_constant<int, kFarCapped>{});
  return a.softcap > 0.f ? capped(std::integral_constant<int, kCapped>{}) : capped(std::integral_constant<int, kUncapped>{});
}

}  // namespace

void attn_tc_box(int* box_d, int* box_l) { *box_d = 64, *box_l = kTile; }

cudaError_t launch_attn_tc(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const AttnArgs& given, int sms,
                           cudaStream_t s) {
  AttnArgs a = given;
  TcScore& x = a.tc;
  x.gain = a.scale * kLog2e;
  x.cap_in = a.softcap > 0.f ? a.scale / a.softcap : 0.f, x.cap_out = a.softcap * kLog2e;
  float power = x.gain;
  for (int i = 0; i < 4; ++i, power *= x.cap_in * x.cap_in) x.poly[i] = kTanh[i] * power;
  // The polynomial is for finite s^2 and coefficients. Where scale / softcap is so large that they are not, the exact
  // form serves for all scores, those of 0 too: reach is NaN.
  x.reach = std::isfinite(x.poly[3]) ? std::fmax(x.cap_in, kTanhRange * 0x1p-60f) : NAN;
  if (a.dk <= 64) return a.dv <= 64 ? launch_shape<1, 1>(q, k, v, a, sms, s) : launch_shape<1, 2>(q, k, v, a, sms, s);
  return a.dv <= 64 ? launch_shape<2, 1>(q, k, v, a, sms, s) : launch_shape<2, 2>(q, k, v, a, sms, s);
}

}  // namespace cb
