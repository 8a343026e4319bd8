// How the decode kernels deal the cache's tokens over the GPU.
//
// An item is one sequence's tokens [first, length) for the query heads of one
// key head (at most a kernel's head count of them).  Items are cut at
// absolute multiples of kDecodeTile tokens, and the tiles of all items, in
// order of (sequence, item), are dealt to the CTAs in equal runs: a CTA walks
// the end of one item, whole items, and the start of another.  Whatever the
// lengths, every CTA reads about the same share of the cache, and only the
// item a run starts or ends inside needs joining: two partial results per CTA.
//
// To begin an item costs a CTA a few microseconds in which it streams nothing
// (lengths, page table, queries and first tokens are read one after another),
// so an item's start counts as decode_item_cost tiles when runs are cut: a run
// through short sequences holds fewer tokens. 64 sequences of 130 to 4000
// tokens, 8 key heads of 128: 115 us without, 106, 98 and 95 with 1, 2 and 3
// bf16 tiles; 8 sequences of 8192 to 16384 fp32 tokens, 12 key heads of 64: 127 without, 112, 119 and 131.
#pragma once

#include "attention_common.cuh"

namespace cb {

constexpr int kDecodeTile = 64;
constexpr int kDecodeMaxBatch = 4096;

struct SeqSpan {
  int lo, hi;      // visible tokens
  int t0, tiles;   // first tile, tiles
  int dealt;       // tiles as dealt: an item's start counts as a.item_cost more
  int len;         // query at position len - 1
};
__device__ __forceinline__ SeqSpan seq_span(const DecodeArgs& a, int b) {
  SeqSpan s;
  const long long room = static_cast<long long>(a.cache.max_pages) * a.cache.page_size;
  s.len = static_cast<int>(min(static_cast<long long>(max(a.length[b], 0)), room));
  s.lo = a.first ? max(a.first[b], 0) : 0;
  s.hi = s.len;
  s.t0 = s.lo / kDecodeTile;
  s.tiles = s.lo < s.hi ? (s.hi - 1) / kDecodeTile + 1 - s.t0 : 0;  // hi may be 2^31 - 1
  s.dealt = s.tiles > 0 ? s.tiles + a.item_cost : 0;
  return s;
}

// Exclusive prefix sums of the sequences' tiles into prefix[0..B] (shared
// memory), by every thread of the CTA; ends with a barrier.
__device__ __forceinline__ void tile_prefix(const DecodeArgs& a, unsigned* prefix) {
  __shared__ unsigned warp_sum[32];
  const int tid = threadIdx.x, n = blockDim.x, lane = tid & 31, warp = tid >> 5, warps = n >> 5;
  const int per = (a.B + n - 1) / n, b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  unsigned sum = 0;
  for (int b = b0; b < b1; ++b) sum += seq_span(a, b).dealt;
  unsigned inc = sum;
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned up = __shfl_up_sync(~0u, inc, o);
    if (lane >= o) inc += up;
  }
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  unsigned base = inc - sum;
  for (int w = 0; w < warps; ++w)
    if (w < warp) base += warp_sum[w];
  for (int b = b0; b < b1; ++b) {
    prefix[b] = base;
    base += seq_span(a, b).dealt;
  }
  if (b1 == a.B && b0 < b1) prefix[a.B] = base;
  __syncthreads();
}

// The run of CTA c: tiles [begin, end) of the `total` dealt ones.
struct Run {
  long long total, ctas;
  __device__ __forceinline__ long long begin(long long c) const { return c * total / ctas; }
  // the CTA whose run holds tile x
  __device__ __forceinline__ long long owner(long long x) const {
    long long c = x * ctas / total;
    while (c + 1 < ctas && begin(c + 1) <= x) ++c;
    while (begin(c) > x) --c;
    return c;
  }
};

// The sequence whose tiles hold dealt tile `at`.
__device__ __forceinline__ int find_seq(const DecodeArgs& a, const unsigned* prefix, int per_seq, long long at) {
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (static_cast<long long>(prefix[mid]) * per_seq <= at) lo = mid;
    else hi = mid;
  }
  return lo;
}

// A piece of a run: part or all of one item.
struct Piece {
  int b, item, hk, h0, heads;  // item = key head * chunks + chunk; query heads [h0, h0 + heads)
  int lo, hi, len;             // the sequence's visible tokens; query at position len - 1
  int tile0, tiles;            // absolute tiles of the sequence
  int dealt;                   // what the piece takes of a run
  bool starts, ends;           // holds the item's first / last tile
  long long last;              // dealt index of the item's last tile
};
__device__ __forceinline__ Piece next_piece(const DecodeArgs& a, const unsigned* prefix, int per_seq, long long at,
                                            long long end, int* b) {
  while (static_cast<long long>(prefix[*b + 1]) * per_seq <= at) ++*b;
  const SeqSpan sp = seq_span(a, *b);
  const long long in_seq = at - static_cast<long long>(prefix[*b]) * per_seq;
  Piece p;
  p.b = *b;
  p.item = static_cast<int>(in_seq / sp.dealt);
  const int off = static_cast<int>(in_seq - static_cast<long long>(p.item) * sp.dealt);
  p.dealt = static_cast<int>(min(static_cast<long long>(sp.dealt - off), end - at));
  const int skip = max(off - a.item_cost, 0);  // the item's tiles before this piece
  p.tile0 = sp.t0 + skip;
  p.tiles = max(off + p.dealt - a.item_cost, 0) - skip;
  p.starts = off == 0;
  p.ends = off + p.dealt == sp.dealt;
  p.last = at - off + sp.dealt - 1;
  p.hk = p.item / a.chunks;
  p.h0 = p.hk * a.group + (p.item % a.chunks) * a.item_heads;
  p.heads = min(a.item_heads, (p.hk + 1) * a.group - p.h0);
  p.lo = sp.lo, p.hi = sp.hi, p.len = sp.len;
  return p;
}

// The piece of a CTA that belongs to a cluster of a.split CTAs per item.
__device__ __forceinline__ Piece whole_piece(const DecodeArgs& a, int per_seq) {
  const int all = blockIdx.x / a.split, rank = blockIdx.x % a.split;
  Piece p;
  p.b = all / per_seq;
  p.item = all % per_seq;
  const SeqSpan sp = seq_span(a, p.b);
  const int begin = static_cast<int>(static_cast<long long>(sp.tiles) * rank / a.split);
  p.tiles = static_cast<int>(static_cast<long long>(sp.tiles) * (rank + 1) / a.split) - begin;
  p.tile0 = sp.t0 + begin;
  p.starts = p.ends = a.split == 1;
  p.last = 0;
  p.hk = p.item / a.chunks;
  p.h0 = p.hk * a.group + (p.item % a.chunks) * a.item_heads;
  p.heads = min(a.item_heads, (p.hk + 1) * a.group - p.h0);
  p.lo = sp.lo, p.hi = sp.hi, p.len = sp.len;
  return p;
}

// The same for contiguous rows: columns are (query, head) pairs r = query *
// group + head in the group, a.item_heads of them per item.
__device__ __forceinline__ Piece rows_piece(const DecodeArgs& a, const AttnArgs& rw) {
  const int all = blockIdx.x / a.split, rank = blockIdx.x % a.split;
  const int rows = rw.Lq * a.group, per_seq = a.Hkv * a.chunks;
  Piece p;
  p.b = all / per_seq;
  p.item = all % per_seq;
  p.hk = p.item / a.chunks;
  p.h0 = (p.item % a.chunks) * a.item_heads;
  p.heads = min(a.item_heads, rows - p.h0);
  p.lo = 0;
  p.hi = row_end(rw, seq_rule(rw, p.b), (p.h0 + p.heads - 1) / a.group);
  p.len = p.hi;
  const int tiles = (p.hi + kDecodeTile - 1) / kDecodeTile;
  p.tile0 = static_cast<int>(static_cast<long long>(tiles) * rank / a.split);
  p.tiles = static_cast<int>(static_cast<long long>(tiles) * (rank + 1) / a.split) - p.tile0;
  p.starts = p.ends = a.split == 1;
  p.last = 0;
  return p;
}

// Sequences without a visible token: zeros, dealt over the CTAs.
template <typename Store>
__device__ __forceinline__ void zero_empty(const DecodeArgs& a, const unsigned* prefix, Store store) {
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    if (prefix[b + 1] != prefix[b]) continue;
    for (int e = threadIdx.x; e < a.Hq * a.dv; e += blockDim.x) store(b * a.os_b + e / a.dv * a.os_h + e % a.dv);
  }
}

// The CTA that starts an item it does not finish says so, for the join.
__device__ __forceinline__ void note_item(const DecodeArgs& a, const Run& run, const Piece& p, int per_seq, long long cta) {
  a.record[2 * cta] = p.b * per_seq + p.item;
  a.record[2 * cta + 1] = static_cast<int>(run.owner(p.last) - cta + 1);
}

// Floats of one partial result: per head m, l, then dv unnormalised sums.
__host__ __device__ inline size_t part_floats(int heads, int dv) { return static_cast<size_t>(heads) * (dv + 2); }

// The page that entry pg of sequence b names, or -1 (and the error recorded).
__device__ __forceinline__ int checked_page(const DecodeArgs& a, int b, int pg) {
  const int page = a.cache.table[b * a.cache.table_stride + pg];
  if (page < 0 || page >= a.cache.num_pages) {
    atomicCAS(a.err, 0, 1);  // CB_ERR_INVALID_ARG
    return -1;
  }
  return page;
}
// Where token j of sequence b lies: its page, or -1 (and the error recorded).
__device__ __forceinline__ int token_page(const DecodeArgs& a, int b, int j, int* slot) {
  const int pg = j / a.cache.page_size;
  *slot = j - pg * a.cache.page_size;
  return checked_page(a, b, pg);
}

}  // namespace cb
