// Host-side checks of views that the attention operators' entry points share.
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <utility>

#include "cb.h"
#include "host_util.h"

namespace cb {

constexpr int kMaxDim = 128;
constexpr int kMaxBatch = 4096;

inline size_t elem_bytes(cb_dtype t) { return t == CB_DTYPE_BF16 ? 2 : 4; }

inline bool heads_ok(const cb_heads* t) {
  if (!t || (t->dtype != CB_DTYPE_F32 && t->dtype != CB_DTYPE_BF16)) return false;
  if (t->batch < 0 || t->len < 0 || t->heads < 1 || t->dim < 1) return false;
  if (t->stride_b < 0 || t->stride_l < 0 || t->stride_h < 0) return false;
  return t->data || t->batch == 0 || t->len == 0;
}

inline bool empty(const cb_heads* t) { return t->batch == 0 || t->len == 0; }

inline bool elem_aligned(const void* p, cb_dtype t) { return reinterpret_cast<uintptr_t>(p) % elem_bytes(t) == 0; }

// Every head's row is made of whole 16-byte pieces at 16-byte boundaries.
inline bool pieces16(const void* data, cb_dtype dt, int dim, long long s0, long long s1, long long s2) {
  const long long per = 16 / static_cast<long long>(elem_bytes(dt));
  return reinterpret_cast<uintptr_t>(data) % 16 == 0 && dim % per == 0 && s0 % per == 0 && s1 % per == 0 && s2 % per == 0;
}
inline bool pieces16(const cb_heads* t) { return pieces16(t->data, t->dtype, t->dim, t->stride_b, t->stride_l, t->stride_h); }

// The bytes of a view: batch x len x heads rows of `row` bytes.
struct Region {
  uintptr_t at;
  int batch, len, heads;
  long long row, sb, sl, sh;  // bytes
  bool empty() const { return batch == 0 || len == 0; }
  // From a token's, a sequence's and the view's first byte to one past its last.
  long long token() const { return (heads - 1LL) * sh + row; }
  long long seq() const { return (len - 1LL) * sl + token(); }
  long long all() const { return (batch - 1LL) * sb + seq(); }
};
inline Region region(const cb_heads* t) {
  const long long e = static_cast<long long>(elem_bytes(t->dtype));
  return {reinterpret_cast<uintptr_t>(t->data), t->batch, t->len, t->heads, t->dim * e, t->stride_b * e, t->stride_l * e, t->stride_h * e};
}

// Whether [0, a) and [d, d + b), both repeated every `period`, stay apart.
inline bool apart(long long period, long long a, long long b, long long d) {
  if (period <= 0 || a > period) return false;
  const long long at = (d % period + period) % period;
  return at >= a && at + b <= period;
}

// Whether two views of the same strides, b's first byte d behind a's, lie with
// their heads' rows between each other's ([..., head, part, dim] buffers): rows
// apart in a token, and a token of both and a sequence of both no wider than
// their strides.
inline bool heads_between(const Region& a, const Region& b, long long d) {
  auto stride = [](int na, long long sa, int nb, long long sb) { return na == 1 ? sb : nb == 1 || sa == sb ? sa : -1LL; };
  const long long sh = stride(a.heads, a.sh, b.heads, b.sh), sl = stride(a.len, a.sl, b.len, b.sl), sb = stride(a.batch, a.sb, b.batch, b.sb);
  if (sh <= 0 || !apart(sh, a.row, b.row, d)) return false;
  auto both = [&](long long in_a, long long in_b) { return std::max(in_a, d + in_b) - std::min(0LL, d); };
  if ((a.len > 1 || b.len > 1) && both(a.token(), b.token()) > sl) return false;
  return (a.batch == 1 && b.batch == 1) || both(a.seq(), b.seq()) <= sb;
}

// True if the views may share a byte. Views whose ranges interleave share none
// if one's rows or sequences lie in the gaps between the other's, at the same
// strides (slices of a wider buffer), or one lies in a single gap.
inline bool overlap(const Region& a, const Region& b) {
  if (a.empty() || b.empty()) return false;
  const long long d = static_cast<long long>(b.at - a.at);
  if (d >= a.all() || -d >= b.all()) return false;
  if (heads_between(a, b, d)) return false;
  auto rows_repeat = [](const Region& t) { return t.batch == 1 || (t.sl > 0 && t.sb % t.sl == 0); };
  if (a.sl == b.sl && rows_repeat(a) && rows_repeat(b) && apart(a.sl, a.token(), b.token(), d)) return false;
  if (a.sb == b.sb && apart(a.sb, a.seq(), b.seq(), d)) return false;
  return !apart(a.sb, a.seq(), b.all(), d) && !apart(b.sb, b.seq(), a.all(), -d);
}
inline bool overlap(const cb_heads* a, const cb_heads* b) { return overlap(region(a), region(b)); }

// Whether no two rows of a view share a byte, as far as its strides nest: each
// at least what the smaller ones span.  For views that are written.
inline bool rows_apart(const Region& r) {
  std::pair<long long, long long> axis[3] = {{r.sb, r.batch}, {r.sl, r.len}, {r.sh, r.heads}};
  std::sort(axis, axis + 3);
  long long span = r.row;
  for (const auto& x : axis) {
    if (x.second <= 1) continue;
    if (x.first < span) return false;
    span += (x.second - 1) * x.first;
  }
  return true;
}

inline bool same_view(const cb_heads* a, const cb_heads* b) {
  return a->data == b->data && a->batch == b->batch && a->len == b->len && a->heads == b->heads && a->dim == b->dim &&
         a->stride_b == b->stride_b && a->stride_l == b->stride_l && a->stride_h == b->stride_h && a->dtype == b->dtype;
}

inline cb_status done(cudaError_t e) { return e == cudaSuccess ? CB_OK : host_cuda_fail(e); }

inline bool score_ok(float scale, float softcap) {
  return std::isfinite(scale) && scale > 0.f && std::isfinite(softcap) && softcap >= 0.f;
}

// The cap as the kernels take it (0: none), away from the ends of fp32's range, where scale / softcap or
// softcap * log2(e) would be 0 or infinite. From 2^100 on a cap moves no score below 2^88 by a bit; below 2^-30
// every weight e^(+-softcap) is 1 in 32 bits, as it is at 2^-30.
inline float kernel_cap(float softcap) {
  if (softcap == 0.f || softcap >= 0x1p100f) return 0.f;
  return softcap < 0x1p-30f ? 0x1p-30f : softcap;
}

}  // namespace cb
