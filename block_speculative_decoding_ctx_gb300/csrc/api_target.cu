// C ABI of the target's side of a cycle: paged cache, attention over it, logit
// adjustment.  See include/dflash.h for the contract of every entry point.
#include <cmath>
#include <cstdint>
#include <cstring>

#include "common.cuh"
#include "paged.h"

using namespace dfl;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int check_cache(const dflash_paged_cache* c) {
  if (!c) return DFLASH_ERR_ARG;
  if (c->format != DFLASH_CACHE_BF16 && c->format != DFLASH_CACHE_F16 && c->format != DFLASH_CACHE_E4M3)
    return DFLASH_ERR_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return DFLASH_ERR_UNSUPPORTED;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
    return DFLASH_ERR_UNSUPPORTED;
  if (c->n_pages < 1 || c->n_kv_heads < 1 || c->n_kv_heads > 4096) return DFLASH_ERR_SHAPE;
  const long long page = (long long)c->n_kv_heads * c->page_size * c->head_dim;
  const int cell = c->format == DFLASH_CACHE_E4M3 ? 1 : 2;
  if (!c->k_pages || !c->v_pages) return DFLASH_ERR_ARG;
  if (c->k_page_stride < page || c->v_page_stride < page || c->k_page_stride > (1ll << 38) ||
      c->v_page_stride > (1ll << 38))
    return DFLASH_ERR_SHAPE;
  if (!aligned(c->k_pages, 16) || !aligned(c->v_pages, 16) || c->k_page_stride * cell % 16 ||
      c->v_page_stride * cell % 16)
    return DFLASH_ERR_ALIGN;
  if (c->format == DFLASH_CACHE_E4M3) {
    if (!c->k_scale || !c->v_scale) return DFLASH_ERR_ARG;
    if (!aligned(c->k_scale, 16) || !aligned(c->v_scale, 16)) return DFLASH_ERR_ALIGN;
  }
  return DFLASH_OK;
}

bool same_cache(const dflash_paged_cache& a, const dflash_paged_cache& b) {
  return a.k_pages == b.k_pages && a.v_pages == b.v_pages && a.k_scale == b.k_scale && a.v_scale == b.v_scale &&
         a.k_page_stride == b.k_page_stride && a.v_page_stride == b.v_page_stride && a.n_pages == b.n_pages &&
         a.n_kv_heads == b.n_kv_heads && a.page_size == b.page_size && a.head_dim == b.head_dim && a.format == b.format;
}

int check_batch(const dflash_paged_batch* b, const dflash_paged_cache* c) {
  if (!b) return DFLASH_ERR_ARG;
  if (b->B < 1 || b->B > 65535 || b->max_pages < 1 || b->rows < 0 || b->rows > (1 << 30)) return DFLASH_ERR_SHAPE;
  if ((long long)b->max_pages * c->page_size >= (1ll << 30) || b->table_stride < b->max_pages) return DFLASH_ERR_SHAPE;
  if (!b->row_start || !b->kv_len || !b->page_table) return DFLASH_ERR_ARG;
  if (!aligned(b->row_start, 4) || !aligned(b->kv_len, 8) || !aligned(b->page_table, 4)) return DFLASH_ERR_ALIGN;
  return DFLASH_OK;
}

// written: every (row, head) has its own place, heads of a row behind one
// another or rows of a head.
int check_rows(const dflash_rows* r, int rows, int heads, int head_dim, bool written) {
  if (!r) return DFLASH_ERR_ARG;
  if (rows == 0) return DFLASH_OK;  // nothing is read or written
  if (!r->ptr) return DFLASH_ERR_ARG;
  if (r->row_stride < 0 || r->head_stride < 0 || (heads > 1 && r->head_stride < head_dim) ||
      (rows > 1 && r->row_stride < head_dim))
    return DFLASH_ERR_SHAPE;
  if (r->row_stride > (1ll << 40) || r->head_stride > (1ll << 40)) return DFLASH_ERR_SHAPE;
  if (!aligned(r->ptr, 16) || r->row_stride % 8 || r->head_stride % 8) return DFLASH_ERR_ALIGN;
  if (written && rows > 1 && heads > 1 && r->row_stride < (heads - 1) * r->head_stride + head_dim &&
      (r->head_stride - head_dim) / r->row_stride < rows - 1)
    return DFLASH_ERR_SHAPE;
  return DFLASH_OK;
}

int check_type(int type, int format) {
  if (type != DFLASH_TYPE_BF16 && type != DFLASH_TYPE_F16) return DFLASH_ERR_ARG;
  if (format == DFLASH_CACHE_BF16 && type != DFLASH_TYPE_BF16) return DFLASH_ERR_ARG;
  if (format == DFLASH_CACHE_F16 && type != DFLASH_TYPE_F16) return DFLASH_ERR_ARG;
  return DFLASH_OK;
}

PagedBatch batch_args(const dflash_paged_batch* b, const dflash_paged_cache* c) {
  PagedBatch p;
  p.row_start = b->row_start;
  p.kv_len = b->kv_len;
  p.table = b->page_table;
  p.table_stride = b->table_stride;
  p.B = b->B;
  p.max_pages = b->max_pages;
  p.rows = b->rows;
  p.n_pages = c->n_pages;
  p.page_shift = 0;
  while ((1 << p.page_shift) < c->page_size) ++p.page_shift;
  return p;
}

int check_workspace(const void* ws, size_t bytes, size_t need) {
  return !ws || !aligned(ws, 256) || bytes < need ? DFLASH_ERR_WORKSPACE : DFLASH_OK;
}

int move(bool append, const dflash_paged_cache* cache, const dflash_paged_batch* batch, int type,
         const dflash_rows* k, const dflash_rows* v, void* workspace, size_t ws_bytes, dflash_stream_t stream) {
  int rc = check_cache(cache);
  if (rc) return rc;
  if ((rc = check_batch(batch, cache))) return rc;
  if ((rc = check_type(type, cache->format))) return rc;
  if ((rc = check_rows(k, batch->rows, cache->n_kv_heads, cache->head_dim, !append))) return rc;
  if ((rc = check_rows(v, batch->rows, cache->n_kv_heads, cache->head_dim, !append))) return rc;
  if ((rc = check_workspace(workspace, ws_bytes, kWsHeader))) return rc;
  PagedMoveArgs a;
  a.batch = batch_args(batch, cache);
  const dflash_rows* x[2] = {k, v};
  for (int i = 0; i < 2; ++i) {
    a.x[i] = static_cast<uint8_t*>(x[i]->ptr);
    a.row_stride[i] = x[i]->row_stride;
    a.head_stride[i] = x[i]->head_stride;
  }
  a.pages[0] = static_cast<uint8_t*>(cache->k_pages);
  a.pages[1] = static_cast<uint8_t*>(cache->v_pages);
  a.scale[0] = cache->k_scale;
  a.scale[1] = cache->v_scale;
  a.page_stride[0] = cache->k_page_stride;
  a.page_stride[1] = cache->v_page_stride;
  a.n_kv = cache->n_kv_heads;
  a.status = static_cast<int*>(workspace);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return append ? launch_paged_append(a, cache->head_dim, cache->format, type, s)
                : launch_paged_gather(a, cache->head_dim, cache->format, type, s);
}

}  // namespace

extern "C" {

int dflash_paged_cache_maps(const dflash_paged_cache* cache, dflash_paged_maps* maps) {
  int rc = check_cache(cache);
  if (rc) return rc;
  if (!maps) return DFLASH_ERR_ARG;
  PagedMaps m = {};
  m.cache = *cache;
  m.cache.maps = nullptr;
  if ((rc = encode_paged_maps(*cache, &m.k, &m.v))) return rc;
  std::memcpy(maps, &m, sizeof(m));
  return DFLASH_OK;
}

size_t dflash_paged_workspace_bytes(void) { return kWsHeader; }

int dflash_paged_append(const dflash_paged_cache* cache, const dflash_paged_batch* batch, int type,
                        const dflash_rows* k, const dflash_rows* v, void* workspace, size_t ws_bytes,
                        dflash_stream_t stream) {
  return move(true, cache, batch, type, k, v, workspace, ws_bytes, stream);
}

int dflash_paged_gather(const dflash_paged_cache* cache, const dflash_paged_batch* batch, int type,
                        const dflash_rows* k, const dflash_rows* v, void* workspace, size_t ws_bytes,
                        dflash_stream_t stream) {
  return move(false, cache, batch, type, k, v, workspace, ws_bytes, stream);
}

size_t dflash_paged_attention_workspace_bytes(int n_q_heads, int n_kv_heads, int head_dim, int max_rows) {
  if (n_q_heads < 1 || n_kv_heads < 1 || n_q_heads % n_kv_heads || max_rows < 0 || (head_dim != 64 && head_dim != 128))
    return 0;
  return paged_attention_workspace(n_q_heads, n_kv_heads, head_dim, max_rows);
}

int dflash_paged_attention(const dflash_paged_cache* cache, const dflash_paged_batch* batch, int type,
                           int n_q_heads, const dflash_rows* q, const dflash_rows* out, float* lse,
                           int max_rows, float scale, int causal, int window, void* workspace,
                           size_t ws_bytes, dflash_stream_t stream) {
  int rc = check_cache(cache);
  if (rc) return rc;
  if ((rc = check_batch(batch, cache))) return rc;
  if ((rc = check_type(type, cache->format))) return rc;
  if (n_q_heads < 1 || n_q_heads % cache->n_kv_heads || n_q_heads > 65535) return DFLASH_ERR_SHAPE;
  const int group = n_q_heads / cache->n_kv_heads;
  if (max_rows < 0 || max_rows > batch->rows || (long long)max_rows * group > (1ll << 30)) return DFLASH_ERR_SHAPE;
  // key tiles of an item, over all KV heads, are counted in 32 bits
  if (((long long)batch->max_pages * cache->page_size / 128 + 16) * cache->n_kv_heads > 0x7FFFFFFFll)
    return DFLASH_ERR_SHAPE;
  if (!(scale > 0.0f) || !std::isfinite(scale * 1.44269504f) || (causal != 0 && causal != 1) || window < 0)
    return DFLASH_ERR_ARG;
  if ((rc = check_rows(q, batch->rows, n_q_heads, cache->head_dim, false))) return rc;
  if ((rc = check_rows(out, batch->rows, n_q_heads, cache->head_dim, true))) return rc;
  if (lse && !aligned(lse, 4)) return DFLASH_ERR_ALIGN;
  if ((rc = check_workspace(workspace, ws_bytes,
                            paged_attention_workspace(n_q_heads, cache->n_kv_heads, cache->head_dim, max_rows))))
    return rc;
  PagedMaps maps;
  if (cache->maps) {
    std::memcpy(&maps, cache->maps, sizeof(maps));
    if (!same_cache(maps.cache, *cache)) return DFLASH_ERR_ARG;
  }
  if (max_rows == 0) return DFLASH_OK;
  if (!cache->maps && (rc = encode_paged_maps(*cache, &maps.k, &maps.v))) return rc;
  PagedAttnArgs a;
  a.batch = batch_args(batch, cache);
  a.k_scale = cache->k_scale;
  a.v_scale = cache->v_scale;
  a.q = static_cast<const uint8_t*>(q->ptr);
  a.out = static_cast<uint8_t*>(out->ptr);
  a.q_row = q->row_stride;
  a.q_head = q->head_stride;
  a.o_row = out->row_stride;
  a.o_head = out->head_stride;
  a.lse = lse;
  a.n_q = n_q_heads;
  a.n_kv = cache->n_kv_heads;
  a.group = group;
  a.max_rows = max_rows;
  a.causal = causal;
  a.window = window < (1 << 30) ? window : 0;  // longer than any position: none
  a.scale_log2 = scale * 1.4426950408889634f;
  a.status = static_cast<int*>(workspace);
  return launch_paged_attention(maps.k, maps.v, a, cache->head_dim, cache->format, type, workspace,
                                reinterpret_cast<cudaStream_t>(stream));
}

size_t dflash_logits_adjust_workspace_bytes(void) { return kWsHeader; }

int dflash_logits_adjust(int B, int G, int vocab, int type, const void* logits, long long l_b, long long l_i,
                         float* out, long long o_b, long long o_i, const dflash_logit_rules* rules,
                         void* workspace, size_t ws_bytes, dflash_stream_t stream) {
  if (B < 1 || G < 1 || G > 64 || (long long)B * G > 65535 || vocab < 1 || vocab > (1 << 18)) return DFLASH_ERR_SHAPE;
  if (type != DFLASH_TYPE_F32 && type != DFLASH_TYPE_BF16 && type != DFLASH_TYPE_F16) return DFLASH_ERR_ARG;
  if (!logits || !out || !rules) return DFLASH_ERR_ARG;
  const dflash_logit_rules& r = *rules;
  if ((r.counts || r.prompt_mask) && r.slots < 1) return DFLASH_ERR_SHAPE;
  if (r.bias_start && r.n_bias < 0) return DFLASH_ERR_SHAPE;
  if (r.bias_start && r.n_bias > 0 && (!r.bias_ids || !r.bias_vals)) return DFLASH_ERR_ARG;
  if (r.draft && G < 2) return DFLASH_ERR_SHAPE;
  const size_t size = type == DFLASH_TYPE_F32 ? 4 : 2;
  if (!aligned(logits, size) || !aligned(out, 4)) return DFLASH_ERR_ALIGN;
  const void* words[] = {r.counts, r.prompt_mask, r.req_slot, r.draft, r.repetition, r.frequency, r.presence,
                         r.bias_start, r.bias_ids, r.bias_vals, r.allow};
  for (const void* p : words)
    if (p && !aligned(p, 4)) return DFLASH_ERR_ALIGN;
  const long long most = 1ll << 40;
  if (l_b < 0 || l_i < 0 || o_b < 0 || o_i < 0 || l_b > most || l_i > most || o_b > most || o_i > most)
    return DFLASH_ERR_SHAPE;
  // every row of the output has its own place: rows of one request behind one
  // another, or requests interleaved
  const long long o_span_i = (G - 1) * o_i + vocab, o_span_b = (B - 1) * o_b + vocab;
  const bool by_b = (G == 1 || o_i >= vocab) && (B == 1 || o_b >= o_span_i);
  const bool by_i = (B == 1 || o_b >= vocab) && (G == 1 || o_i >= o_span_b);
  if (!by_b && !by_i) return DFLASH_ERR_SHAPE;
  const bool same = type == DFLASH_TYPE_F32 && logits == out && (B == 1 || l_b == o_b) && (G == 1 || l_i == o_i);
  const char* l0 = static_cast<const char*>(logits);
  const char* l1 = l0 + ((B - 1) * l_b + (G - 1) * l_i + vocab) * size;
  const char* o0 = reinterpret_cast<const char*>(out);
  const char* o1 = o0 + ((B - 1) * o_b + (G - 1) * o_i + vocab) * 4;
  if (!same && l0 < o1 && o0 < l1) return DFLASH_ERR_ARG;
  int rc = check_workspace(workspace, ws_bytes, kWsHeader);
  if (rc) return rc;
  LogitsArgs a;
  a.logits = logits;
  a.out = out;
  a.l_b = l_b;
  a.l_i = l_i;
  a.o_b = o_b;
  a.o_i = o_i;
  a.B = B;
  a.G = G;
  a.V = vocab;
  a.r = r;
  a.status = static_cast<int*>(workspace);
  return launch_logits_adjust(a, type, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
