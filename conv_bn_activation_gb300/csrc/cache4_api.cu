// Entry points of the head norms and rotations and of the 4-bit cache: argument
// validation, kernel choice and launches.  Host code only.
#include <initializer_list>

#include "cb.h"
#include "host_util.h"
#include "internal.h"
#include "views.h"

using namespace cb;

namespace {

constexpr int kMaxAxes = 8;
constexpr int kMaxHeads = 65536;  // heads times dims, items and lanes' words are counted in 32 bits

long long code_bytes(int dim) { return (dim + 1) / 2; }
long long scale_bytes(int dim) { return 4LL * ((dim + 63) / 64); }

// The four arrays of a cache's pages: keys' codes and scales, values' codes and scales.
struct Pages4 {
  Region part[4];
};
Pages4 pages(const cb_paged_cache4* c) {
  auto at = [&](const void* p, long long row, long long sp, long long st, long long sh, long long unit) {
    return Region{reinterpret_cast<uintptr_t>(p), c->num_pages, c->page_size, c->heads, row, sp * unit, st * unit, sh * unit};
  };
  return {{at(c->k, code_bytes(c->dim_k), c->k_stride_page, c->k_stride_slot, c->k_stride_head, 1),
           at(c->k_scale, scale_bytes(c->dim_k), c->ks_stride_page, c->ks_stride_slot, c->ks_stride_head, 2),
           at(c->v, code_bytes(c->dim_v), c->v_stride_page, c->v_stride_slot, c->v_stride_head, 1),
           at(c->v_scale, scale_bytes(c->dim_v), c->vs_stride_page, c->vs_stride_slot, c->vs_stride_head, 2)}};
}

bool cache_ok(const cb_paged_cache4* c) {
  if (!c) return false;
  if (c->num_pages < 0 || c->page_size < 1 || c->heads < 1 || c->dim_k < 1 || c->dim_v < 1) return false;
  if (c->batch < 0 || c->max_pages < 0 || c->table_stride < 0) return false;
  if (static_cast<long long>(c->max_pages) * c->page_size >= (1LL << 31)) return false;
  for (const long long s : {c->k_stride_page, c->k_stride_slot, c->k_stride_head, c->v_stride_page, c->v_stride_slot,
                            c->v_stride_head, c->ks_stride_page, c->ks_stride_slot, c->ks_stride_head, c->vs_stride_page,
                            c->vs_stride_slot, c->vs_stride_head})
    if (s < 0) return false;
  if (c->num_pages > 0 && (!c->k || !c->v || !c->k_scale || !c->v_scale)) return false;
  return c->table || c->batch == 0 || c->max_pages == 0;
}

bool aligned(const cb_paged_cache4* c) {
  return reinterpret_cast<uintptr_t>(c->k_scale) % 2 == 0 && reinterpret_cast<uintptr_t>(c->v_scale) % 2 == 0;
}

// Rows of whole pieces of `piece` bytes of codes, and a row's scales one word: what the streaming kernels copy, at
// offsets of 32 bits in those units.
bool pieces(const cb_paged_cache4* c, int piece, const void* codes, const void* scales, int dim, std::initializer_list<long long> code_strides,
            std::initializer_list<long long> scale_strides) {
  const int unit = dim <= 64 ? 2 : 4;
  auto reach = [&](const std::initializer_list<long long>& s, long long per) {  // of pages, slots and heads
    const double last = static_cast<double>(s.begin()[0]) * c->num_pages + static_cast<double>(s.begin()[1]) * c->page_size +
                        static_cast<double>(s.begin()[2]) * c->heads;
    return last / static_cast<double>(per) < 4294967296.0;
  };
  if (!reach(code_strides, piece) || !reach(scale_strides, unit)) return false;
  if (dim % (2 * piece) != 0 || reinterpret_cast<uintptr_t>(codes) % piece != 0 || reinterpret_cast<uintptr_t>(scales) % (2 * unit) != 0)
    return false;
  for (const long long s : code_strides)
    if (s % piece != 0) return false;
  for (const long long s : scale_strides)
    if (s % unit != 0) return false;
  return true;
}
// The largest pieces that rows of keys and values are made of: 16 bytes, 4 or none.
int pieces(const cb_paged_cache4* c) {
  if (c->num_pages == 0) return 0;
  for (const int piece : {16, 4})
    if (pieces(c, piece, c->k, c->k_scale, c->dim_k, {c->k_stride_page, c->k_stride_slot, c->k_stride_head},
               {c->ks_stride_page, c->ks_stride_slot, c->ks_stride_head}) &&
        pieces(c, piece, c->v, c->v_scale, c->dim_v, {c->v_stride_page, c->v_stride_slot, c->v_stride_head},
               {c->vs_stride_page, c->vs_stride_slot, c->vs_stride_head}))
      return piece;
  return 0;
}

// Tokens and pages that the kernels for whole words take: rows of 16-byte pieces, dims that are multiples of 8, heads
// within 32 bits of their token's or slot's first.
bool words(const cb_heads* t, const void* codes, int dim, long long page, long long slot, long long head, long long scale_head) {
  auto near = [&](long long stride) { return stride * (t->heads - 1) + dim < (1LL << 31); };
  return dim % 8 == 0 && pieces16(t) && reinterpret_cast<uintptr_t>(codes) % 4 == 0 && page % 4 == 0 && slot % 4 == 0 &&
         head % 4 == 0 && near(t->stride_h) && near(head) && near(scale_head);
}
bool words(const cb_heads* k, const cb_heads* v, const cb_paged_cache4* c) {
  return words(k, c->k, c->dim_k, c->k_stride_page, c->k_stride_slot, c->k_stride_head, c->ks_stride_head) &&
         words(v, c->v, c->dim_v, c->v_stride_page, c->v_stride_slot, c->v_stride_head, c->vs_stride_head);
}

// The codes' pages as the streaming kernels' copies take them; false where they cannot.
bool code_map(CUtensorMap* m, const void* codes, const cb_paged_cache4* c, int dim, long long page, long long slot, long long head) {
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(dim / 2), static_cast<cuuint64_t>(c->page_size), static_cast<cuuint64_t>(c->heads),
                              static_cast<cuuint64_t>(c->num_pages)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(slot), static_cast<cuuint64_t>(head), static_cast<cuuint64_t>(page)};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(decode4_box(c->dim_k, c->dim_v)), 16, 1, 1};
  return host_map_u8(m, codes, dims, strides, box);
}

bool overlap(const cb_heads* t, const cb_paged_cache4* c) {
  for (const Region& r : pages(c).part)
    if (cb::overlap(r, region(t))) return true;
  return false;
}

PagedArgs paged_args(const cb_paged_cache4* c) {
  PagedArgs p{};
  p.k = c->k, p.v = c->v;
  p.ks_p = c->k_stride_page, p.ks_t = c->k_stride_slot, p.ks_h = c->k_stride_head;
  p.vs_p = c->v_stride_page, p.vs_t = c->v_stride_slot, p.vs_h = c->v_stride_head;
  p.k_scale = static_cast<const uint16_t*>(c->k_scale), p.v_scale = static_cast<const uint16_t*>(c->v_scale);
  p.kx_p = c->ks_stride_page, p.kx_t = c->ks_stride_slot, p.kx_h = c->ks_stride_head;
  p.vx_p = c->vs_stride_page, p.vx_t = c->vs_stride_slot, p.vx_h = c->vs_stride_head;
  p.table = c->table;
  p.table_stride = c->table_stride;
  p.num_pages = c->num_pages, p.page_size = c->page_size, p.max_pages = c->max_pages;
  return p;
}

// Tokens of a call and the cache they belong to.
cb_status check_tokens(const cb_heads* k, const cb_heads* v, const cb_paged_cache4* cache) {
  if (!heads_ok(k) || !heads_ok(v) || !cache_ok(cache)) return CB_ERR_INVALID_ARG;
  if (k->batch != cache->batch || v->batch != cache->batch || k->len != v->len) return CB_ERR_INVALID_ARG;
  if (k->heads != cache->heads || v->heads != cache->heads) return CB_ERR_INVALID_ARG;
  if (k->dim != cache->dim_k || v->dim != cache->dim_v || k->dtype != v->dtype) return CB_ERR_INVALID_ARG;
  if (cache->dim_k > kMaxDim || cache->dim_v > kMaxDim || cache->heads > kMaxHeads) return CB_ERR_UNSUPPORTED;
  if (!elem_aligned(k->data, k->dtype) || !elem_aligned(v->data, v->dtype) || !aligned(cache)) return CB_ERR_ALIGNMENT;
  return CB_OK;
}

cb_status check_decode(const cb_heads* q, const cb_paged_cache4* cache) {
  if (!heads_ok(q) || !cache_ok(cache)) return CB_ERR_INVALID_ARG;
  if (q->len != 1 || q->batch != cache->batch || q->dim != cache->dim_k || q->heads % cache->heads != 0) return CB_ERR_INVALID_ARG;
  if (cache->dim_k > kMaxDim || cache->dim_v > kMaxDim || q->batch > kMaxBatch || q->heads > kMaxHeads) return CB_ERR_UNSUPPORTED;
  return CB_OK;
}

struct Decode4Plan {
  int sms = 0, ctas = 0, chunks = 0, heads = 0, split = 0;
  int* err = nullptr;
  int piece = 0;
};
cb_status plan_decode(const cb_heads* q, const cb_paged_cache4* cache, Decode4Plan* p) {
  const cb_status st = host_device(&p->sms, &p->err);
  if (st != CB_OK) return st;
  p->piece = pieces(cache);
  const bool bf16 = q->dtype == CB_DTYPE_BF16;
  const int group = q->heads / cache->heads, most = !p->piece ? kDecodeSimtHeads : bf16 ? kDecode4Heads : kDecode4HeadsF32;
  p->chunks = (group + most - 1) / most;
  p->heads = (group + p->chunks - 1) / p->chunks;
  p->ctas = p->sms * (p->piece ? decode4_ctas_per_sm(cache->dim_k, cache->dim_v, bf16, p->heads, q->batch) : 4);
  // Whole items on clusters where a CTA then walks at most 16 tiles, as for other caches (cb_attention_decode).
  const long long items = static_cast<long long>(q->batch) * cache->heads * p->chunks;
  const long long tiles = (static_cast<long long>(cache->max_pages) * cache->page_size + 63) / 64;
  p->split = 1;
  while (p->split < 8 && items * p->split * 2 <= p->ctas && p->split < tiles) p->split *= 2;
  if (!p->piece || tiles > 16LL * p->split) p->split = 0;
  return CB_OK;
}

}  // namespace

extern "C" {

cb_status cb_norm_rotate(const cb_heads* q, const cb_heads* k, const cb_head_rule* rule, cb_heads* q_out, cb_heads* k_out,
                         void* stream) {
  if (!heads_ok(q) || !heads_ok(q_out) || !rule || (k == nullptr) != (k_out == nullptr)) return CB_ERR_INVALID_ARG;
  if (k && (!heads_ok(k) || !heads_ok(k_out))) return CB_ERR_INVALID_ARG;
  const cb_heads* in[2] = {q, k};
  cb_heads* out[2] = {q_out, k_out};
  const int views = k ? 2 : 1;
  for (int i = 0; i < views; ++i) {
    if (in[i]->batch != q->batch || in[i]->len != q->len || in[i]->dim != q->dim || in[i]->dtype != q->dtype) return CB_ERR_INVALID_ARG;
    if (out[i]->batch != q->batch || out[i]->len != q->len || out[i]->dim != q->dim || out[i]->dtype != q->dtype) return CB_ERR_INVALID_ARG;
    if (out[i]->heads != in[i]->heads || !rows_apart(region(out[i]))) return CB_ERR_INVALID_ARG;
    for (int j = 0; j < views; ++j)
      if (!(i == j && same_view(in[i], out[i])) && overlap(out[i], in[j])) return CB_ERR_INVALID_ARG;
  }
  if (k && overlap(q_out, k_out)) return CB_ERR_INVALID_ARG;
  if (rule->norm && !(rule->eps >= 0.f && std::isfinite(rule->eps))) return CB_ERR_INVALID_ARG;
  if (rule->rotary < 0 || rule->rotary > q->dim || rule->rotary % 2 != 0) return CB_ERR_INVALID_ARG;
  if (rule->axes < 1 || rule->axes > kMaxAxes || rule->pos_stride_axis < 0 || rule->pos_stride_b < 0) return CB_ERR_INVALID_ARG;
  if (rule->rotary > 0 && (!rule->freq || (!rule->pos && !empty(q)))) return CB_ERR_INVALID_ARG;
  if (q->dim > kMaxDim || static_cast<long long>(q->batch) * q->len >= (1LL << 31)) return CB_ERR_UNSUPPORTED;
  if (q->heads > kMaxHeads || (k && k->heads > kMaxHeads)) return CB_ERR_UNSUPPORTED;
  for (int i = 0; i < views; ++i)
    if (!elem_aligned(in[i]->data, q->dtype) || !elem_aligned(out[i]->data, q->dtype)) return CB_ERR_ALIGNMENT;
  if (empty(q)) return CB_OK;
  RotateArgs a{};
  int sms = 0;
  const cb_status st = host_device(&sms, &a.err);
  if (st != CB_OK) return st;
  for (int i = 0; i < views; ++i) {
    RotateView& v = a.v[i];
    v.x = in[i]->data, v.y = out[i]->data;
    v.xs_b = in[i]->stride_b, v.xs_l = in[i]->stride_l, v.xs_h = in[i]->stride_h;
    v.ys_b = out[i]->stride_b, v.ys_l = out[i]->stride_l, v.ys_h = out[i]->stride_h;
    v.weight = !rule->norm ? nullptr : i == 0 ? rule->q_weight : rule->k_weight;
    v.heads = in[i]->heads;
  }
  a.B = q->batch, a.L = q->len, a.dim = q->dim, a.rotary = rule->rotary;
  a.adjacent = rule->adjacent != 0, a.norm = rule->norm != 0, a.axes = rule->axes, a.eps = rule->eps;
  a.freq = rule->freq, a.axis = rule->axis, a.pos = rule->pos;
  a.ps_a = rule->pos_stride_axis, a.ps_b = rule->pos_stride_b;
  return done(launch_norm_rotate(a, q->dtype == CB_DTYPE_BF16, sms, static_cast<cudaStream_t>(stream)));
}

cb_status cb_cache4_append(const cb_heads* k_new, const cb_heads* v_new, const int* pos, const int* count,
                           const cb_paged_cache4* cache, void* stream) {
  cb_status st = check_tokens(k_new, v_new, cache);
  if (st != CB_OK) return st;
  if (empty(k_new)) return CB_OK;
  if (!pos || overlap(k_new, cache) || overlap(v_new, cache)) return CB_ERR_INVALID_ARG;
  AppendArgs a{};
  int sms = 0;
  st = host_device(&sms, &a.err);
  if (st != CB_OK) return st;
  a.k = k_new->data, a.v = v_new->data;
  a.ks_b = k_new->stride_b, a.ks_l = k_new->stride_l, a.ks_h = k_new->stride_h;
  a.vs_b = v_new->stride_b, a.vs_l = v_new->stride_l, a.vs_h = v_new->stride_h;
  a.pos = pos, a.count = count;
  a.cache = paged_args(cache);
  a.B = k_new->batch, a.T = k_new->len, a.H = cache->heads, a.dk = cache->dim_k, a.dv = cache->dim_v;
  return done(launch_cache4_append(a, k_new->dtype == CB_DTYPE_BF16, words(k_new, v_new, cache), sms, static_cast<cudaStream_t>(stream)));
}

cb_status cb_cache4_read(const cb_paged_cache4* cache, const int* first, const int* count, cb_heads* k_out, cb_heads* v_out,
                         void* stream) {
  cb_status st = check_tokens(k_out, v_out, cache);
  if (st != CB_OK) return st;
  if (empty(k_out)) return CB_OK;
  if (overlap(k_out, cache) || overlap(v_out, cache) || overlap(k_out, v_out)) return CB_ERR_INVALID_ARG;
  if (!rows_apart(region(k_out)) || !rows_apart(region(v_out))) return CB_ERR_INVALID_ARG;
  Read4Args a{};
  int sms = 0;
  st = host_device(&sms, &a.err);
  if (st != CB_OK) return st;
  a.k = k_out->data, a.v = v_out->data;
  a.ks_b = k_out->stride_b, a.ks_l = k_out->stride_l, a.ks_h = k_out->stride_h;
  a.vs_b = v_out->stride_b, a.vs_l = v_out->stride_l, a.vs_h = v_out->stride_h;
  a.first = first, a.count = count;
  a.cache = paged_args(cache);
  a.B = k_out->batch, a.T = k_out->len, a.H = cache->heads, a.dk = cache->dim_k, a.dv = cache->dim_v;
  return done(launch_cache4_read(a, k_out->dtype == CB_DTYPE_BF16, words(k_out, v_out, cache), sms, static_cast<cudaStream_t>(stream)));
}

cb_status cb_attention_decode4_workspace(const cb_heads* q, const cb_paged_cache4* cache, size_t* bytes) {
  if (!bytes) return CB_ERR_INVALID_ARG;
  cb_status st = check_decode(q, cache);
  if (st != CB_OK) return st;
  Decode4Plan p;
  st = plan_decode(q, cache, &p);
  if (st != CB_OK) return st;
  *bytes = decode_workspace_bytes(p.ctas, p.heads, cache->dim_v);
  return CB_OK;
}

cb_status cb_attention_decode4(const cb_heads* q, const cb_paged_cache4* cache, const int* length, const int* first,
                               float scale, float softcap, const float* slopes, cb_heads* out, void* workspace,
                               size_t workspace_bytes, void* stream) {
  cb_status st = check_decode(q, cache);
  if (st != CB_OK && st != CB_ERR_UNSUPPORTED) return st;
  if (!heads_ok(out) || out->len != 1 || out->batch != q->batch || out->heads != q->heads || out->dim != cache->dim_v ||
      out->dtype != q->dtype || overlap(out, q) || !rows_apart(region(out)) || !score_ok(scale, softcap))
    return CB_ERR_INVALID_ARG;
  if (st != CB_OK) return st;
  if (!elem_aligned(q->data, q->dtype) || !elem_aligned(out->data, q->dtype) || !aligned(cache)) return CB_ERR_ALIGNMENT;
  if (q->batch == 0) return CB_OK;
  if (!length || !workspace || overlap(out, cache)) return CB_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(workspace) % 256 != 0) return CB_ERR_ALIGNMENT;
  Decode4Plan p;
  st = plan_decode(q, cache, &p);
  if (st != CB_OK) return st;
  if (workspace_bytes < decode_workspace_bytes(p.ctas, p.heads, cache->dim_v)) return CB_ERR_WORKSPACE;
  DecodeArgs a{};
  a.q = q->data, a.o = out->data;
  a.qs_b = q->stride_b, a.qs_h = q->stride_h, a.os_b = out->stride_b, a.os_h = out->stride_h;
  a.cache = paged_args(cache);
  a.length = length, a.first = first, a.slopes = slopes;
  a.scale = scale, a.softcap = kernel_cap(softcap);
  a.B = q->batch, a.Hq = q->heads, a.Hkv = cache->heads, a.group = q->heads / cache->heads;
  a.dk = cache->dim_k, a.dv = cache->dim_v;
  a.chunks = p.chunks, a.item_heads = p.heads, a.split = p.split;
  a.item_cost = decode4_item_cost(q->dtype == CB_DTYPE_BF16);
  a.record = static_cast<int*>(workspace);
  a.part = reinterpret_cast<float*>(a.record + 2 * p.ctas);
  a.ctas = p.ctas;
  a.err = p.err;
  a.timeout_ns = host_timeout_ns();
  Maps4 maps;
  const bool mapped = p.piece == 16 && !p.split && cache->num_pages > 0 && cache->page_size % 16 == 0 &&
                      code_map(&maps.k, cache->k, cache, cache->dim_k, cache->k_stride_page, cache->k_stride_slot, cache->k_stride_head) &&
                      code_map(&maps.v, cache->v, cache, cache->dim_v, cache->v_stride_page, cache->v_stride_slot, cache->v_stride_head);
  return done(launch_decode4(a, q->dtype == CB_DTYPE_BF16, p.piece, mapped ? &maps : nullptr, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
