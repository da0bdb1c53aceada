// echo_kv_api.hip -- the C ABI of the quantized K/V cache declared in
// include/echo.h: argument validation, marshalling and launch.  Every check
// runs before the first HIP call.
#include <math.h>
#include <stdint.h>

#include "echo.h"
#include "echo_kv_internal.h"

using namespace echo;

namespace {

constexpr int64_t kMaxThreads = 0xffffffffll;        // work-items of a dispatch along x
constexpr int64_t kMaxSeqs = 65535;
constexpr int32_t kMaxRows = 1 << 30;                // row and position indices stay inside 31 bits

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_buf(const void* p) {
  if (!p) return ECHO_ERR_ARG;
  return aligned16(p) ? ECHO_OK : ECHO_ERR_ALIGN;
}

int check_form(const echo_kv_cache* c) {
  if (!c) return ECHO_ERR_ARG;
  if (c->bits != 4 && c->bits != 8) return ECHO_ERR_ARG;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return ECHO_ERR_ARG;
  if (c->group != 32 && c->group != 64 && c->group != 128) return ECHO_ERR_ARG;
  if (c->group > c->head_dim) return ECHO_ERR_ARG;
  if (c->kv_heads < 1 || c->kv_heads > 4096) return ECHO_ERR_ARG;
  if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1))) return ECHO_ERR_ARG;
  if (c->num_pages < 1 || c->num_pages > INT32_MAX) return ECHO_ERR_SHAPE;
  return ECHO_OK;
}

int check_cache(const echo_kv_cache* c) {
  int rc;
  if ((rc = check_form(c))) return rc;
  const void* bufs[] = {c->k_codes, c->v_codes, c->k_params, c->v_params};
  for (const void* p : bufs)
    if ((rc = check_buf(p))) return rc;
  return ECHO_OK;
}

int check_batch_sizes(const echo_kv_batch* b) {
  if (!b) return ECHO_ERR_ARG;
  if (b->seqs < 0 || b->rows < 0 || b->max_new < 0 || b->max_len < 0 || b->table_stride < 0) return ECHO_ERR_SHAPE;
  if (b->seqs > kMaxSeqs || b->rows > kMaxRows || b->max_new > kMaxRows || b->max_len > kMaxRows ||
      b->table_stride > kMaxRows)
    return ECHO_ERR_SHAPE;
  return ECHO_OK;
}

// Device index arrays: int32, read element by element.
int check_index(const void* p) {
  if (!p) return ECHO_ERR_ARG;
  return (reinterpret_cast<uintptr_t>(p) & 3u) ? ECHO_ERR_ALIGN : ECHO_OK;
}

int check_batch(const echo_kv_batch* b) {
  int rc;
  if ((rc = check_index(b->row_start)) || (rc = check_index(b->kv_len))) return rc;
  return b->table_stride ? check_index(b->page_table) : ECHO_OK;
}

// Rows [rows, heads, D]: D contiguous, every row 16-byte aligned.  `out`:
// no two rows may share an element.
int check_rows(const echo_kv_rows* r, int64_t rows, int64_t heads, int64_t D, bool f32, bool out) {
  int rc;
  if (!r) return ECHO_ERR_ARG;
  if (r->dtype != ECHO_KV_BF16 && r->dtype != ECHO_KV_F16 && !(f32 && r->dtype == ECHO_KV_F32)) return ECHO_ERR_ARG;
  if ((rc = check_buf(r->data))) return rc;
  const int64_t rs = r->row_stride, hs = r->head_stride;
  const int64_t most = (int64_t)1 << 40;    // elements from the first row to the last one, more than any memory
  if (rs < 0 || hs < 0 || rs > most || hs > most) return ECHO_ERR_ARG;
  if ((rows > 1 && rs > most / (rows - 1)) || (heads > 1 && hs > most / (heads - 1))) return ECHO_ERR_ARG;
  const int64_t unit = r->dtype == ECHO_KV_F32 ? 4 : 8;
  if ((rows > 1 && rs % unit) || (heads > 1 && hs % unit)) return ECHO_ERR_ALIGN;
  if (out) {
    // (rows - 1) * rs and (heads - 1) * hs are at most `most` each
    const bool row_major = (heads == 1 || hs >= D) && (rows == 1 || rs >= (heads - 1) * hs + D);
    const bool head_major = (rows == 1 || rs >= D) && (heads == 1 || hs >= (rows - 1) * rs + D);
    if (!row_major && !head_major) return ECHO_ERR_ARG;
  }
  return ECHO_OK;
}

KvCache cache_of(const echo_kv_cache* c) {
  KvCache k;
  k.k_codes = static_cast<uint8_t*>(c->k_codes);
  k.v_codes = static_cast<uint8_t*>(c->v_codes);
  k.k_params = c->k_params;
  k.v_params = c->v_params;
  k.num_pages = c->num_pages;
  k.bits = c->bits;
  k.group = c->group;
  k.head_dim = c->head_dim;
  k.kv_heads = c->kv_heads;
  k.page_shift = __builtin_ctz((unsigned)c->page_size);
  return k;
}

KvBatch batch_of(const echo_kv_batch* b) {
  KvBatch k;
  k.row_start = b->row_start;
  k.kv_len = b->kv_len;
  k.page_table = b->page_table;
  k.table_stride = b->table_stride;
  k.seqs = b->seqs;
  k.rows = b->rows;
  k.max_new = b->max_new < b->rows ? b->max_new : b->rows;
  k.max_len = b->max_len;
  return k;
}

KvRows rows_of(const echo_kv_rows* r) { return KvRows{r->data, r->row_stride, r->head_stride, r->dtype}; }

int launched(hipError_t e) { return e == hipSuccess ? ECHO_OK : ECHO_ERR_HIP; }

// Options and sizes of an attention call; *empty: there is no row to compute.
int check_attention(const echo_kv_cache* c, const echo_kv_batch* b, int q_heads, int causal, int window, int sinks,
                    bool* empty, KvPlan* plan) {
  int rc;
  if ((rc = check_form(c)) || (rc = check_batch_sizes(b))) return rc;
  if (q_heads < c->kv_heads || q_heads % c->kv_heads || q_heads > (1 << 20)) return ECHO_ERR_ARG;
  if ((causal != 0 && causal != 1) || window < 0 || sinks < 0) return ECHO_ERR_ARG;
  if (window > 0 && !causal) return ECHO_ERR_ARG;
  if (sinks > 0 && window == 0) return ECHO_ERR_ARG;
  *empty = b->rows == 0 || b->seqs == 0 || b->max_new == 0;
  if (*empty) return ECHO_OK;
  const int per = q_heads / c->kv_heads;
  const KvBatch k = batch_of(b);
  if ((int64_t)k.max_new * per > (int64_t)1 << 30) return ECHO_ERR_SHAPE;
  *plan = kv_attention_plan(cache_of(c), k, per, causal, window, sinks);
  const int64_t most = kMaxThreads / kv_plan_threads(*plan) / plan->splits;
  if ((int64_t)c->kv_heads * b->seqs * plan->row_blocks > most) return ECHO_ERR_SHAPE;
  return ECHO_OK;
}

// Workspace of an attention call whose keys are split: kKvCounters counters,
// the same for every call so that calls of any sizes can take turns with it,
// the splits' outputs in fp32, and their (maximum, sum) pairs.
int64_t part_rows(const echo_kv_cache* c, const echo_kv_batch* b, const KvPlan& p) {
  return p.splits > 1 ? (int64_t)b->seqs * c->kv_heads * kv_plan_rows(p) * p.splits : 0;
}
size_t workspace_bytes_of(int64_t part_rows, int head_dim) {
  return part_rows ? ((size_t)kKvCounters + (size_t)part_rows * (head_dim + 2)) * 4 : 0;
}

int cache_rows(const echo_kv_cache* cache, const echo_kv_batch* batch, const echo_kv_rows* k, const echo_kv_rows* v,
               bool out, KvWriteArgs* a) {
  int rc;
  if ((rc = check_form(cache)) || (rc = check_batch_sizes(batch))) return rc;
  if (!k || !v) return ECHO_ERR_ARG;
  if (k->dtype != v->dtype) return ECHO_ERR_ARG;
  if (kv_cache_blocks(cache_of(cache), batch_of(batch)) > kMaxThreads / kKvCacheThreads) return ECHO_ERR_SHAPE;
  if (batch->rows == 0 || batch->seqs == 0) return ECHO_OK;
  if ((rc = check_cache(cache)) || (rc = check_batch(batch))) return rc;
  if ((rc = check_rows(k, batch->rows, cache->kv_heads, cache->head_dim, true, out))) return rc;
  if ((rc = check_rows(v, batch->rows, cache->kv_heads, cache->head_dim, true, out))) return rc;
  if (out && k->data == v->data) return ECHO_ERR_ARG;
  a->c = cache_of(cache);
  a->b = batch_of(batch);
  a->k = rows_of(k);
  a->v = rows_of(v);
  return ECHO_OK;
}

}  // namespace

extern "C" {

int echo_kv_write(const echo_kv_cache* cache, const echo_kv_batch* batch, const echo_kv_rows* k, const echo_kv_rows* v,
                  void* stream) {
  KvWriteArgs a;
  const int rc = cache_rows(cache, batch, k, v, false, &a);
  if (rc || batch->rows == 0 || batch->seqs == 0) return rc;
  return launched(run_kv_write(a, static_cast<hipStream_t>(stream)));
}

int echo_kv_read(const echo_kv_cache* cache, const echo_kv_batch* batch, const echo_kv_rows* k, const echo_kv_rows* v,
                 void* stream) {
  KvWriteArgs a;
  const int rc = cache_rows(cache, batch, k, v, true, &a);
  if (rc || batch->rows == 0 || batch->seqs == 0) return rc;
  return launched(run_kv_read(a, static_cast<hipStream_t>(stream)));
}

int echo_kv_attention(const echo_kv_cache* cache, const echo_kv_batch* batch, int q_heads, const echo_kv_rows* q,
                      const echo_kv_rows* out, float scale, int causal, int window, int sinks, void* workspace,
                      size_t workspace_bytes, void* stream) {
  int rc;
  bool empty;
  KvAttnArgs a;
  if ((rc = check_attention(cache, batch, q_heads, causal, window, sinks, &empty, &a.plan))) return rc;
  if (!isfinite(scale) || !q || !out || q->dtype != out->dtype) return ECHO_ERR_ARG;
  if (empty) return ECHO_OK;
  if ((rc = check_cache(cache)) || (rc = check_batch(batch))) return rc;
  if ((rc = check_rows(q, batch->rows, q_heads, cache->head_dim, false, false))) return rc;
  if ((rc = check_rows(out, batch->rows, q_heads, cache->head_dim, false, true))) return rc;
  const int64_t parts = part_rows(cache, batch, a.plan);
  if (parts) {
    if ((rc = check_buf(workspace))) return rc;
    if (workspace_bytes < workspace_bytes_of(parts, cache->head_dim)) return ECHO_ERR_ARG;
  }
  a.c = cache_of(cache);
  a.b = batch_of(batch);
  a.q = rows_of(q);
  a.out = rows_of(out);
  a.heads_per_kv = q_heads / cache->kv_heads;
  a.scale_log2 = (float)frexp((double)scale * 1.4426950408889634, &a.scale_exp);   // the product may pass FLT_MAX
  a.causal = causal;
  a.window = window;
  a.sinks = sinks;
  a.counters = static_cast<uint32_t*>(workspace);
  a.part_o = static_cast<float*>(workspace) + kKvCounters;
  a.part_ml = a.part_o + parts * cache->head_dim;
  return launched(run_kv_attention(a, static_cast<hipStream_t>(stream)));
}

size_t echo_kv_codes_bytes(const echo_kv_cache* c) {
  if (check_form(c)) return 0;
  return (size_t)c->num_pages * c->kv_heads * c->page_size * (c->head_dim * c->bits / 8);
}

size_t echo_kv_params_bytes(const echo_kv_cache* c) {
  if (check_form(c)) return 0;
  return (size_t)c->num_pages * c->kv_heads * c->page_size * (c->head_dim / c->group) * sizeof(uint32_t);
}

size_t echo_kv_workspace_bytes(const echo_kv_cache* cache, const echo_kv_batch* batch, int q_heads, int causal,
                               int window, int sinks) {
  bool empty;
  KvPlan plan;
  if (check_attention(cache, batch, q_heads, causal, window, sinks, &empty, &plan) || empty) return 0;
  return workspace_bytes_of(part_rows(cache, batch, plan), cache->head_dim);
}

}  // extern "C"
