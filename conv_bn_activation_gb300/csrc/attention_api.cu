// Entry points of the attention operators: argument validation, kernel choice
// and launches.  Host code only.
#include "cb.h"
#include "host_util.h"
#include "internal.h"
#include "views.h"

using namespace cb;

namespace {

bool cache_ok(const cb_paged_cache* c) {
  if (!c || (c->dtype != CB_DTYPE_F32 && c->dtype != CB_DTYPE_BF16)) return false;
  if (c->num_pages < 0 || c->page_size < 1 || c->heads < 1 || c->dim_k < 1 || c->dim_v < 1) return false;
  if (c->batch < 0 || c->max_pages < 0 || c->table_stride < 0) return false;
  if (static_cast<long long>(c->max_pages) * c->page_size >= (1LL << 31)) return false;
  if (c->k_stride_page < 0 || c->k_stride_slot < 0 || c->k_stride_head < 0) return false;
  if (c->v_stride_page < 0 || c->v_stride_slot < 0 || c->v_stride_head < 0) return false;
  if (c->num_pages > 0 && (!c->k || !c->v)) return false;
  return c->table || c->batch == 0 || c->max_pages == 0;
}

bool pieces16(const cb_paged_cache* c) {
  return cb::pieces16(c->k, c->dtype, c->dim_k, c->k_stride_page, c->k_stride_slot, c->k_stride_head) &&
         cb::pieces16(c->v, c->dtype, c->dim_v, c->v_stride_page, c->v_stride_slot, c->v_stride_head);
}

// Whether a view may share an element with the cache's pages.
bool overlap(const cb_heads* t, const cb_paged_cache* c) {
  const cb_heads k{c->k, c->num_pages, c->page_size, c->heads, c->dim_k, c->k_stride_page, c->k_stride_slot, c->k_stride_head, c->dtype};
  const cb_heads v{c->v, c->num_pages, c->page_size, c->heads, c->dim_v, c->v_stride_page, c->v_stride_slot, c->v_stride_head, c->dtype};
  return cb::overlap(&k, t) || cb::overlap(&v, t);
}

PagedArgs paged_args(const cb_paged_cache* c) {
  PagedArgs p{};
  p.k = c->k, p.v = c->v;
  p.ks_p = c->k_stride_page, p.ks_t = c->k_stride_slot, p.ks_h = c->k_stride_head;
  p.vs_p = c->v_stride_page, p.vs_t = c->v_stride_slot, p.vs_h = c->v_stride_head;
  p.table = c->table;
  p.table_stride = c->table_stride;
  p.num_pages = c->num_pages, p.page_size = c->page_size, p.max_pages = c->max_pages;
  return p;
}

// The tensor-core kernel's map of a view: (dim, heads, len, batch).
bool tc_map(CUtensorMap* m, const cb_heads* t) {
  int box_d = 0, box_l = 0;
  attn_tc_box(&box_d, &box_l);
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(t->dim), static_cast<cuuint64_t>(t->heads),
                              static_cast<cuuint64_t>(t->len), static_cast<cuuint64_t>(t->batch)};
  const cuuint64_t strides[3] = {2 * static_cast<cuuint64_t>(t->stride_h), 2 * static_cast<cuuint64_t>(t->stride_l),
                                 2 * static_cast<cuuint64_t>(t->stride_b)};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(box_d), 1, static_cast<cuuint32_t>(box_l), 1};
  return host_map_bf16(m, t->data, dims, strides, box);
}

// Whether the streaming kernel (columns of at most 16 or 8 (query, head) pairs,
// keys split over clusters) beats the tiled one of its dtype.
// bf16: the tiled kernel walks pairs of 128-row tiles, mostly empty rows when
// there are few queries, and cannot split the keys.  32 sequences, 4 key heads,
// groups of 5, 2048 keys: 8 queries 54 against 78 us, 16 queries 90 against 78;
// one sequence, 2 heads, 2048 keys, 64 queries: 11 against 22 us.
// fp32: an item of 8 columns reads all its keys anew, and costs the GPU about
// 1.3e-4 us per key; a wave of tiles of 64 rows takes 0.12 us per key however
// few they are: 900 items per wave (32 heads on 4, 512 keys: 64 queries of one
// sequence 26 against 62 us, 16 of 8 sequences 41 and 63, 64 of 8 136 and 85).
// An item's start counts as 120 keys, a tile's as 50 (7 sequences of 82 tokens,
// 10 heads on 2: 33 against 23 us; 4 of 160, 8 on 2: 22 and 29).
bool few_queries(const AttnArgs& a, bool bf16, int sms) {
  const long long rows = static_cast<long long>(a.Lq) * a.group;
  if (!bf16) {
    const long long seqs = static_cast<long long>(a.B) * (a.Hq / a.group), waves = ((rows + 63) / 64 * seqs + 2 * sms - 1) / (2 * sms);
    return (rows + kDecodeSimtHeads - 1) / kDecodeSimtHeads * seqs * (a.Lk + 120) <= 6 * sms * waves * (a.Lk + 50);
  }
  const long long chunks = (rows + kDecodeMmaHeads - 1) / kDecodeMmaHeads;
  const long long pairs = (static_cast<long long>((a.Lq + 127) / 128) * a.group + 1) / 2;
  return 2 * chunks <= 3 * pairs || (chunks <= 8 && a.Lk >= 256 && 4 * pairs * a.B * (a.Hq / a.group) <= sms);
}

// Shapes of a decode call; fills nothing it refuses.
cb_status check_decode(const cb_heads* q, const cb_paged_cache* cache) {
  if (!heads_ok(q) || !cache_ok(cache)) return CB_ERR_INVALID_ARG;
  if (q->len != 1 || q->batch != cache->batch || q->dim != cache->dim_k || q->dtype != cache->dtype ||
      q->heads % cache->heads != 0)
    return CB_ERR_INVALID_ARG;
  if (cache->dim_k > kMaxDim || cache->dim_v > kMaxDim || q->batch > kMaxBatch) return CB_ERR_UNSUPPORTED;
  return CB_OK;
}

struct DecodePlan {
  int sms = 0, ctas = 0, chunks = 0, heads = 0, split = 0;
  int* err = nullptr;
  bool vec = false;
};
cb_status plan_decode(const cb_heads* q, const cb_paged_cache* cache, DecodePlan* p) {
  const cb_status st = host_device(&p->sms, &p->err);
  if (st != CB_OK) return st;
  p->vec = pieces16(cache);
  const bool mma = q->dtype == CB_DTYPE_BF16 && p->vec;
  // One wave of resident CTAs: their runs are equal, so a second wave would only add pieces to join.
  const int group = q->heads / cache->heads, most = mma ? kDecodeMmaHeads : kDecodeSimtHeads;
  p->chunks = (group + most - 1) / most;
  p->heads = (group + p->chunks - 1) / p->chunks;
  p->ctas = p->sms * (p->vec ? decode_ctas_per_sm(cache->dim_k, cache->dim_v, mma, p->heads, q->batch) : 4);
  // Whole items on clusters where that leaves a CTA at most 16 tiles of 64
  // tokens of the largest cache the table can name: no join then, and no CTA
  // walks much longer than another.  Else runs.  (61 sequences of 944 to 2729
  // tokens, 2 key heads of 64: 17.5 us, as runs 22; for more tiles see decode_stream.cuh.)
  const long long items = static_cast<long long>(q->batch) * cache->heads * p->chunks;
  const long long tiles = (static_cast<long long>(cache->max_pages) * cache->page_size + 63) / 64;
  p->split = 1;
  while (p->split < 8 && items * p->split * 2 <= p->ctas && p->split < tiles) p->split *= 2;
  if (!p->vec || tiles > 16LL * p->split) p->split = 0;
  return CB_OK;
}

}  // namespace

extern "C" {

cb_status cb_attention(const cb_heads* q, const cb_heads* k, const cb_heads* v, const cb_score* score, cb_heads* out,
                       void* stream) {
  if (!heads_ok(q) || !heads_ok(k) || !heads_ok(v) || !heads_ok(out) || !score) return CB_ERR_INVALID_ARG;
  if (k->batch != q->batch || v->batch != q->batch || out->batch != q->batch) return CB_ERR_INVALID_ARG;
  if (v->len != k->len || out->len != q->len || out->heads != q->heads || v->heads != k->heads) return CB_ERR_INVALID_ARG;
  if (q->heads % k->heads != 0 || k->dim != q->dim || out->dim != v->dim) return CB_ERR_INVALID_ARG;
  if (k->dtype != q->dtype || v->dtype != q->dtype || out->dtype != q->dtype) return CB_ERR_INVALID_ARG;
  if (!score_ok(score->scale, score->softcap)) return CB_ERR_INVALID_ARG;
  if (score->q_offset > (1 << 29) || score->q_offset < -(1 << 29)) return CB_ERR_INVALID_ARG;
  if (score->prefix_len && !score->causal) return CB_ERR_INVALID_ARG;
  if (k->len > 0 && (score->doc_q == nullptr) != (score->doc_k == nullptr)) return CB_ERR_INVALID_ARG;
  if (overlap(out, q) || overlap(out, k) || overlap(out, v)) return CB_ERR_INVALID_ARG;
  if (q->dim > kMaxDim || v->dim > kMaxDim || q->len > (1 << 29) || k->len > (1 << 29)) return CB_ERR_UNSUPPORTED;
  for (const cb_heads* t : {q, k, v, static_cast<const cb_heads*>(out)})
    if (!elem_aligned(t->data, t->dtype)) return CB_ERR_ALIGNMENT;
  if (empty(q)) return CB_OK;
  if (static_cast<long long>(q->batch) * q->heads * ((q->len + 31) / 32) >= (1LL << 31)) return CB_ERR_UNSUPPORTED;
  if (static_cast<long long>(q->len) * (q->heads / k->heads) > (1LL << 31) - 256) return CB_ERR_UNSUPPORTED;  // rows of a key head
  AttnArgs a{};
  int sms = 0;
  const cb_status st = host_device(&sms, &a.err);
  if (st != CB_OK) return st;
  a.q = q->data, a.k = k->data, a.v = v->data, a.o = out->data;
  a.qs_b = q->stride_b, a.qs_l = q->stride_l, a.qs_h = q->stride_h;
  a.ks_b = k->stride_b, a.ks_l = k->stride_l, a.ks_h = k->stride_h;
  a.vs_b = v->stride_b, a.vs_l = v->stride_l, a.vs_h = v->stride_h;
  a.os_b = out->stride_b, a.os_l = out->stride_l, a.os_h = out->stride_h;
  a.B = q->batch, a.Lq = q->len, a.Lk = k->len, a.Hq = q->heads, a.group = q->heads / k->heads;
  a.dk = q->dim, a.dv = v->dim;
  a.scale = score->scale, a.softcap = kernel_cap(score->softcap), a.slopes = score->slopes;
  a.causal = score->causal ? 1 : 0, a.q_offset = score->q_offset;
  a.prefix_len = score->prefix_len, a.kv_len = score->kv_len;
  if (k->len > 0) a.doc_q = score->doc_q, a.doc_k = score->doc_k;
  a.timeout_ns = host_timeout_ns();
  const bool vec = pieces16(q) && pieces16(k) && pieces16(v) && pieces16(out);
  if (vec && few_queries(a, q->dtype == CB_DTYPE_BF16, sms))
    return done(launch_attn_rows(a, q->dtype == CB_DTYPE_BF16, sms, static_cast<cudaStream_t>(stream)));
  CUtensorMap qm, km, vm;
  if (q->dtype == CB_DTYPE_BF16 && vec && k->len >= 1 && k->len <= kAttnTcMaxKeys && tc_map(&qm, q) && tc_map(&km, k) &&
      tc_map(&vm, v))
    return done(launch_attn_tc(qm, km, vm, a, sms, static_cast<cudaStream_t>(stream)));
  return done(launch_attn_simt(a, q->dtype == CB_DTYPE_BF16, vec, sms, static_cast<cudaStream_t>(stream)));
}

cb_status cb_cache_append(const cb_heads* k_new, const cb_heads* v_new, const int* pos, const int* count,
                          const cb_paged_cache* cache, void* stream) {
  if (!heads_ok(k_new) || !heads_ok(v_new) || !cache_ok(cache)) return CB_ERR_INVALID_ARG;
  if (k_new->batch != cache->batch || v_new->batch != cache->batch || k_new->len != v_new->len) return CB_ERR_INVALID_ARG;
  if (k_new->heads != cache->heads || v_new->heads != cache->heads) return CB_ERR_INVALID_ARG;
  if (k_new->dim != cache->dim_k || v_new->dim != cache->dim_v) return CB_ERR_INVALID_ARG;
  if (k_new->dtype != cache->dtype || v_new->dtype != cache->dtype) return CB_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(k_new->data), static_cast<const void*>(v_new->data),
                        static_cast<const void*>(cache->k), static_cast<const void*>(cache->v)})
    if (!elem_aligned(p, cache->dtype)) return CB_ERR_ALIGNMENT;
  if (empty(k_new)) return CB_OK;
  if (!pos || overlap(k_new, cache) || overlap(v_new, cache)) return CB_ERR_INVALID_ARG;
  AppendArgs a{};
  int sms = 0;
  const cb_status st = host_device(&sms, &a.err);
  if (st != CB_OK) return st;
  a.k = k_new->data, a.v = v_new->data;
  a.ks_b = k_new->stride_b, a.ks_l = k_new->stride_l, a.ks_h = k_new->stride_h;
  a.vs_b = v_new->stride_b, a.vs_l = v_new->stride_l, a.vs_h = v_new->stride_h;
  a.pos = pos, a.count = count;
  a.cache = paged_args(cache);
  a.B = k_new->batch, a.T = k_new->len, a.H = cache->heads, a.dk = cache->dim_k, a.dv = cache->dim_v;
  const int eb = static_cast<int>(elem_bytes(cache->dtype));
  const bool vec = pieces16(k_new) && pieces16(v_new) && pieces16(cache);
  return done(launch_cache_append(a, eb, vec ? 16 : eb, sms, static_cast<cudaStream_t>(stream)));
}

cb_status cb_attention_decode_workspace(const cb_heads* q, const cb_paged_cache* cache, size_t* bytes) {
  if (!bytes) return CB_ERR_INVALID_ARG;
  cb_status st = check_decode(q, cache);
  if (st != CB_OK) return st;
  DecodePlan p;
  st = plan_decode(q, cache, &p);
  if (st != CB_OK) return st;
  *bytes = decode_workspace_bytes(p.ctas, p.heads, cache->dim_v);
  return CB_OK;
}

cb_status cb_attention_decode(const cb_heads* q, const cb_paged_cache* cache, const int* length, const int* first,
                              float scale, float softcap, const float* slopes, cb_heads* out, void* workspace,
                              size_t workspace_bytes, void* stream) {
  cb_status st = check_decode(q, cache);
  if (st != CB_OK && st != CB_ERR_UNSUPPORTED) return st;
  if (!heads_ok(out) || out->len != 1 || out->batch != q->batch || out->heads != q->heads || out->dim != cache->dim_v ||
      out->dtype != q->dtype || overlap(out, q) || !score_ok(scale, softcap))
    return CB_ERR_INVALID_ARG;
  if (st != CB_OK) return st;
  for (const void* p : {static_cast<const void*>(q->data), static_cast<const void*>(out->data),
                        static_cast<const void*>(cache->k), static_cast<const void*>(cache->v)})
    if (!elem_aligned(p, q->dtype)) return CB_ERR_ALIGNMENT;
  if (q->batch == 0) return CB_OK;
  if (!length || !workspace || overlap(out, cache)) return CB_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(workspace) % 256 != 0) return CB_ERR_ALIGNMENT;
  DecodePlan p;
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
  a.item_cost = decode_item_cost(q->dtype == CB_DTYPE_BF16);
  a.record = static_cast<int*>(workspace);
  a.part = reinterpret_cast<float*>(a.record + 2 * p.ctas);
  a.ctas = p.ctas;
  a.err = p.err;
  return done(launch_decode(a, q->dtype == CB_DTYPE_BF16, p.vec, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
