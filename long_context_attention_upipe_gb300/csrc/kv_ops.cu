// C-ABI entry points of the paged cache of keys and values and of the attention that reads it: argument checks
// on the host, then the launches.
#include <cmath>

#include "checks.h"
#include "common.cuh"
#include "internal.h"

using namespace upipe;

namespace {

constexpr int64_t kMaxSpan = (int64_t)1 << 48;  // bytes; keeps every product below in range

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

// Rows of a cache's tensor: [pages][heads][tokens] of `row` bytes, strides in bytes (0 where there is one).
struct PoolRows {
  const void* base;
  int64_t n[3], s[3], row;  // by falling stride
  int64_t span() const { return (n[0] - 1) * s[0] + (n[1] - 1) * s[1] + (n[2] - 1) * s[2] + row; }
};

bool pool_rows(PoolRows& r, const void* base, int64_t pages, int64_t heads, int64_t tokens, int64_t ps, int64_t hs, int64_t ts,
               int64_t elem, int64_t row) {
  r = PoolRows{base, {pages, heads, tokens}, {pages > 1 ? ps : 0, heads > 1 ? hs : 0, tokens > 1 ? ts : 0}, row};
  for (int i = 0; i < 3; ++i) {
    if (r.s[i] < 0 || r.s[i] > kMaxSpan / 16 / r.n[i]) return false;
    r.s[i] *= elem;
    if (r.s[i] >= (int64_t)1 << 40) return false;  // what a TMA map takes
  }
  for (int i = 0; i < 2; ++i)  // sort three by falling stride
    for (int j = 0; j < 2 - i; ++j)
      if (r.s[j] < r.s[j + 1]) {
        std::swap(r.s[j], r.s[j + 1]);
        std::swap(r.n[j], r.n[j + 1]);
      }
  return true;
}

// Bytes that the levels below `level` take up.
int64_t inner_span(const PoolRows& r, int level) {
  int64_t x = r.row;
  for (int i = level + 1; i < 3; ++i) x += (r.n[i] - 1) * r.s[i];
  return x;
}

bool pool_disjoint(const PoolRows& r) {
  for (int i = 0; i < 3; ++i)
    if (r.n[i] > 1 && r.s[i] < inner_span(r, i)) return false;
  return true;
}

// Two tensors of the same shape and strides, rows of either disjoint: whether they share bytes when the second lies `d` bytes behind
// the first.  A row of each meet if some difference of their indices, |i| < n at each level, leaves less than a row of d; what the levels
// below span leaves two differences to look at.
bool meet_at(const PoolRows& r, int level, int64_t d) {
  if (level == 3) return d > -r.row && d < r.row;
  if (r.n[level] <= 1) return meet_at(r, level + 1, d);
  const int64_t s = r.s[level], q = d >= 0 ? d / s : -((s - 1 - d) / s);  // floor
  for (int64_t i = q; i <= q + 1; ++i)
    if (i > -r.n[level] && i < r.n[level] && meet_at(r, level + 1, d - i * s)) return true;
  return false;
}
bool pools_meet(const PoolRows& a, const PoolRows& b) {
  return meet_at(a, 0, reinterpret_cast<intptr_t>(b.base) - reinterpret_cast<intptr_t>(a.base));
}

struct CacheSpans {
  Buf b[4];  // k, v and their scales
};

upipe_status_t check_cache(const upipe_kv_cache_t* c, KvCache& out, CacheSpans& spans) {
  if (!c || !c->k || !c->v || c->n_pages <= 0 || c->n_pages > INT32_MAX || c->page_size <= 0 || c->n_kv_heads <= 0 ||
      c->head_dim <= 0 || (c->dtype != 0 && c->dtype != 1) || !c->k_scale != !c->dtype || !c->v_scale != !c->dtype)
    return UPIPE_ERR_INVALID_ARG;
  if ((c->head_dim != 64 && c->head_dim != 128) || c->page_size % 16 || c->page_size > (1 << 20) || c->n_kv_heads > 1024)
    return UPIPE_ERR_UNSUPPORTED;
  const int elem = c->dtype ? 1 : 2;
  PoolRows r[4];
  for (int i = 0; i < 2; ++i)
    if (!pool_rows(r[i], i ? c->v : c->k, c->n_pages, c->n_kv_heads, c->page_size, c->page_stride, c->head_stride,
                   c->token_stride, elem, c->head_dim * elem))
      return UPIPE_ERR_INVALID_ARG;
  if (c->dtype)
    for (int i = 0; i < 2; ++i)
      if (!pool_rows(r[2 + i], i ? c->v_scale : c->k_scale, c->n_pages, c->n_kv_heads, c->page_size, c->scale_page_stride,
                     c->scale_head_stride, c->scale_token_stride, 4, 4))
        return UPIPE_ERR_INVALID_ARG;
  for (int i = 0; i < (c->dtype ? 4 : 2); i += 2)
    if (!pool_disjoint(r[i]) || pools_meet(r[i], r[i + 1])) return UPIPE_ERR_INVALID_ARG;  // (strides are above zero then)
  for (int i = 0; i < 3; ++i)
    if (r[0].s[i] % 16) return UPIPE_ERR_UNSUPPORTED;
  if (!aligned16(c->k) || !aligned16(c->v) || !aligned16(c->k_scale) || !aligned16(c->v_scale)) return UPIPE_ERR_ALIGNMENT;
  spans = CacheSpans{{{c->k, r[0].span()}, {c->v, r[1].span()}, {nullptr, 0}, {nullptr, 0}}};
  if (c->dtype) {
    spans.b[2] = Buf{c->k_scale, r[2].span()};
    spans.b[3] = Buf{c->v_scale, r[3].span()};
    for (int i = 0; i < 2; ++i)
      for (int j = 2; j < 4; ++j)
        if (overlaps(spans.b[i].p, spans.b[i].bytes, spans.b[j].p, spans.b[j].bytes)) return UPIPE_ERR_INVALID_ARG;
  }
  // strides of a single page, head or token do not count
  const bool pg = c->n_pages > 1, hd = c->n_kv_heads > 1;
  out = KvCache{c->k,
                c->v,
                c->k_scale,
                c->v_scale,
                pg ? c->page_stride : 0,
                hd ? c->head_stride : 0,
                c->token_stride,
                pg ? c->scale_page_stride : 0,
                hd ? c->scale_head_stride : 0,
                c->scale_token_stride,
                (int)c->n_pages,
                c->page_size,
                c->n_kv_heads,
                c->head_dim,
                c->dtype};
  return UPIPE_OK;
}

upipe_status_t check_table(const upipe_page_table_t* t, PageTable& out, Buf& span) {
  if (!t || t->n_seqs < 0 || t->max_pages < 0 || (t->n_seqs > 1 && t->stride < t->max_pages)) return UPIPE_ERR_INVALID_ARG;
  const bool some = t->n_seqs > 0 && t->max_pages > 0;
  if (some && !t->pages) return UPIPE_ERR_INVALID_ARG;
  if (t->n_seqs > 65536) return UPIPE_ERR_UNSUPPORTED;
  if (t->n_seqs > 1 && t->stride > kMaxSpan / 4 / t->n_seqs) return UPIPE_ERR_INVALID_ARG;
  if (!aligned4(t->pages)) return UPIPE_ERR_ALIGNMENT;
  out = PageTable{t->pages, t->n_seqs > 1 ? t->stride : 0, t->n_seqs, t->max_pages};
  span = Buf{some ? t->pages : nullptr, some ? 4 * ((t->n_seqs - 1) * out.stride + t->max_pages) : 0};
  return UPIPE_OK;
}

// Heads of bf16 rows at p with the given strides in elements.
upipe_status_t check_heads(const void* p, int64_t heads, int64_t tokens, int64_t hs, int64_t ts, int head_dim, HeadRows& out) {
  if (!p) return UPIPE_ERR_INVALID_ARG;
  out = rows_of(p, heads, tokens, hs, ts, head_dim);
  if (out.hs < 0 || out.ts < 0 || out.hs > kMaxSpan / 8 / heads || out.ts > kMaxSpan / 8 / tokens) return UPIPE_ERR_INVALID_ARG;
  if (out.hs % 8 || out.ts % 8) return UPIPE_ERR_UNSUPPORTED;
  return aligned16(p) ? UPIPE_OK : UPIPE_ERR_ALIGNMENT;
}

bool apart(const Buf& a, const Buf& b) { return !overlaps(a.p, a.bytes, b.p, b.bytes); }

// Whether a buffer shares no byte with any of the cache's tensors.
bool apart(const Buf& a, const CacheSpans& c) {
  for (const Buf& b : c.b)
    if (!apart(a, b)) return false;
  return true;
}

Buf buf(const HeadRows& r) { return Buf{r.base, r.bytes()}; }

upipe_status_t kv_copy(bool write, const upipe_kv_cache_t* cache, const upipe_page_table_t* table, int64_t tokens,
                       const int32_t* seq, const int32_t* pos, const uint16_t* k, int64_t k_head_stride, int64_t k_token_stride,
                       const uint16_t* v, int64_t v_head_stride, int64_t v_token_stride, void* stream) {
  KvArgs a{};
  CacheSpans spans;
  Buf pages;
  upipe_status_t s = check_cache(cache, a.c, spans);
  if (s == UPIPE_OK) s = check_table(table, a.t, pages);
  if (s != UPIPE_OK) return s;
  if (tokens < 0 || tokens > INT32_MAX) return UPIPE_ERR_INVALID_ARG;
  if (tokens == 0) return UPIPE_OK;
  if (!seq || !pos) return UPIPE_ERR_INVALID_ARG;
  HeadRows kr, vr;
  s = check_heads(k, a.c.n_kv_heads, tokens, k_head_stride, k_token_stride, a.c.head_dim, kr);
  if (s == UPIPE_OK) s = check_heads(v, a.c.n_kv_heads, tokens, v_head_stride, v_token_stride, a.c.head_dim, vr);
  if (s != UPIPE_OK) return s;
  if (!aligned4(seq) || !aligned4(pos)) return UPIPE_ERR_ALIGNMENT;
  const Buf sq{seq, 4 * tokens}, ps{pos, 4 * tokens}, kb = buf(kr), vb = buf(vr);
  if (!apart(kb, spans) || !apart(vb, spans)) return UPIPE_ERR_INVALID_ARG;
  if (write) {
    if (!apart(sq, spans) || !apart(ps, spans) || !apart(pages, spans)) return UPIPE_ERR_INVALID_ARG;
  } else {
    if (!rows_disjoint(kr.heads, tokens, kr.hs, kr.ts, a.c.head_dim) || !rows_disjoint(vr.heads, tokens, vr.hs, vr.ts, a.c.head_dim) ||
        rows_may_meet(kr, vr) || !outputs_apart({kb}, {sq, ps, pages}) || !outputs_apart({vb}, {sq, ps, pages}))
      return UPIPE_ERR_INVALID_ARG;
  }
  auto heads = [](const uint16_t* p, const HeadRows& r) {
    return KvHeads{const_cast<bf16*>(reinterpret_cast<const bf16*>(p)), r.hs, r.ts};
  };
  a.k = heads(k, kr);
  a.v = heads(v, vr);
  a.tokens = tokens;
  a.seq = seq;
  a.pos = pos;
  return finish(write ? launch_kv_write(a, (cudaStream_t)stream) : launch_kv_read(a, (cudaStream_t)stream));
}

upipe_status_t check_queries(const KvCache& c, int32_t n_q_heads, int32_t q_len) {
  if (n_q_heads <= 0 || n_q_heads % c.n_kv_heads || q_len <= 0) return UPIPE_ERR_INVALID_ARG;
  if (q_len > 16 || n_q_heads / c.n_kv_heads > 128) return UPIPE_ERR_UNSUPPORTED;
  return UPIPE_OK;
}

}  // namespace

extern "C" {

upipe_status_t upipe_attn_kv_write(const upipe_kv_cache_t* cache, const upipe_page_table_t* table, int64_t tokens,
                                   const int32_t* seq, const int32_t* pos, const uint16_t* k, int64_t k_head_stride,
                                   int64_t k_token_stride, const uint16_t* v, int64_t v_head_stride, int64_t v_token_stride,
                                   void* stream) {
  return kv_copy(true, cache, table, tokens, seq, pos, k, k_head_stride, k_token_stride, v, v_head_stride, v_token_stride, stream);
}

upipe_status_t upipe_attn_kv_read(const upipe_kv_cache_t* cache, const upipe_page_table_t* table, int64_t tokens,
                                  const int32_t* seq, const int32_t* pos, uint16_t* k, int64_t k_head_stride,
                                  int64_t k_token_stride, uint16_t* v, int64_t v_head_stride, int64_t v_token_stride,
                                  void* stream) {
  return kv_copy(false, cache, table, tokens, seq, pos, k, k_head_stride, k_token_stride, v, v_head_stride, v_token_stride, stream);
}

upipe_status_t upipe_attn_decode_workspace_size(const upipe_kv_cache_t* cache, int32_t n_seqs, int32_t n_q_heads, int32_t q_len,
                                                size_t* bytes) {
  DecodeArgs a{};
  CacheSpans spans;
  upipe_status_t s = check_cache(cache, a.c, spans);
  if (s == UPIPE_OK) s = check_queries(a.c, n_q_heads, q_len);
  if (s != UPIPE_OK) return s;
  if (!bytes || n_seqs < 0) return UPIPE_ERR_INVALID_ARG;
  if (n_seqs > 65536) return UPIPE_ERR_UNSUPPORTED;
  a.t.n_seqs = n_seqs;
  a.q_len = q_len;
  a.hq = n_q_heads;
  *bytes = decode_workspace(a);
  return UPIPE_OK;
}

upipe_status_t upipe_attn_decode(const upipe_kv_cache_t* cache, const upipe_page_table_t* table, const int32_t* lens,
                                 int32_t n_q_heads, int32_t q_len, float softmax_scale, const uint16_t* q,
                                 int64_t q_head_stride, int64_t q_token_stride, uint16_t* o, int64_t o_head_stride,
                                 int64_t o_token_stride, float* lse, void* ws, size_t ws_bytes, void* stream) {
  DecodeArgs a{};
  CacheSpans spans;
  Buf pages;
  upipe_status_t s = check_cache(cache, a.c, spans);
  if (s == UPIPE_OK) s = check_table(table, a.t, pages);
  if (s == UPIPE_OK) s = check_queries(a.c, n_q_heads, q_len);
  if (s != UPIPE_OK) return s;
  if (!std::isfinite(softmax_scale)) return UPIPE_ERR_INVALID_ARG;
  const int64_t tokens = (int64_t)a.t.n_seqs * q_len;
  if (tokens == 0) return UPIPE_OK;
  if (!lens || !ws) return UPIPE_ERR_INVALID_ARG;
  HeadRows qr, orow;
  s = check_heads(q, n_q_heads, tokens, q_head_stride, q_token_stride, a.c.head_dim, qr);
  if (s == UPIPE_OK) s = check_heads(o, n_q_heads, tokens, o_head_stride, o_token_stride, a.c.head_dim, orow);
  if (s != UPIPE_OK) return s;
  if (!aligned4(lens) || !aligned16(lse) || !aligned16(ws)) return UPIPE_ERR_ALIGNMENT;
  a.lens = lens;
  a.hq = n_q_heads;
  a.q_len = q_len;
  const size_t need = decode_workspace(a);
  if (ws_bytes < need) return UPIPE_ERR_WORKSPACE_TOO_SMALL;
  const Buf lb{lens, 4 * (int64_t)a.t.n_seqs}, eb{lse, lse ? 4 * tokens * n_q_heads : 0}, wb{ws, (int64_t)need}, ob = buf(orow);
  if (!rows_disjoint(orow.heads, tokens, orow.hs, orow.ts, a.c.head_dim) || rows_may_meet(qr, orow) ||
      !outputs_apart({eb, wb}, {lb, pages, buf(qr), ob}) || !outputs_apart({ob}, {lb, pages}) || !apart(ob, spans) ||
      !apart(eb, spans) || !apart(wb, spans))
    return UPIPE_ERR_INVALID_ARG;
  a.scale = softmax_scale == 0.f ? 1.f / std::sqrt((float)a.c.head_dim) : softmax_scale;
  a.q = reinterpret_cast<const bf16*>(q);
  a.q_head = qr.hs;
  a.q_tok = qr.ts;
  a.o = reinterpret_cast<bf16*>(o);
  a.o_head = orow.hs;
  a.o_tok = orow.ts;
  a.lse = lse;
  a.ws = ws;
  return finish(launch_decode(a, (cudaStream_t)stream));
}

}  // extern "C"
