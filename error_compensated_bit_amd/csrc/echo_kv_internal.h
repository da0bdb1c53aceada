// echo_kv_internal.h -- types shared by the C-ABI layer and the gfx950 kernels
// of the quantized K/V cache.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace echo {

// element-type tags (same values as the ECHO_KV_* constants of the public header)
constexpr int kKvBF16 = 0, kKvF16 = 1, kKvF32 = 2;

// The cache.  codes: [num_pages][kv_heads][page][D * bits / 8] bytes, params:
// [num_pages][kv_heads][page][D / group] words, for keys and for values.
struct KvCache {
  uint8_t *k_codes, *v_codes;
  uint32_t *k_params, *v_params;
  int64_t num_pages;
  int32_t bits, group, head_dim, kv_heads;
  int32_t page_shift;   // log2 of the page's slots
};

// Which rows a call brings and where they lie (device arrays).
struct KvBatch {
  const int32_t* row_start;    // seqs + 1
  const int32_t* kv_len;       // seqs
  const int32_t* page_table;   // seqs * table_stride
  int64_t table_stride;
  int32_t seqs, rows, max_new, max_len;
};

// 16- or 32-bit rows [rows, heads, D]: element strides, D contiguous.
struct KvRows {
  void* p;
  int64_t row_stride, head_stride;
  int32_t dtype;
};

struct KvWriteArgs {
  KvCache c;
  KvBatch b;
  KvRows k, v;
};

// Arrival counters in a workspace: keys are split only where there are fewer blocks of rows than this.
constexpr int kKvCounters = 256;

// How an attention call is cut into blocks; a function of host arguments only.
struct KvPlan {
  int32_t row_tiles;      // 16-row tiles a wave works on
  int32_t row_waves;      // 1: a block's waves share its rows and take turns over the keys; more: each has its own rows
  int32_t key_waves;      // waves of a block that share rows: 4 or 8
  int32_t row_blocks;     // blocks over the rows of one (sequence, K/V head)
  int32_t splits;         // blocks over the keys
  int32_t split_tiles;    // 32-key tiles of one split
};

struct KvAttnArgs {
  KvCache c;
  KvBatch b;
  KvRows q, out;
  int32_t heads_per_kv;   // query heads that share a K/V head
  float scale_log2;       // softmax scale * log2(e) * 2^-scale_exp: 0, or 1/2 to 1 in size
  int32_t scale_exp;
  int32_t causal, window, sinks;
  KvPlan plan;
  uint32_t* counters;        // arrived splits of every (sequence, K/V head, block of rows); 0 between calls
  float *part_o, *part_ml;   // results of the splits: [seq][K/V head][row][split] of D floats, and (maximum, sum)
};

// Each returns the first launch error (hipSuccess when every launch went out).
hipError_t run_kv_write(const KvWriteArgs& a, hipStream_t st);
hipError_t run_kv_read(const KvWriteArgs& a, hipStream_t st);
// Blocks along x of both, and their threads.
constexpr int kKvCacheThreads = 256;
int64_t kv_cache_blocks(const KvCache& c, const KvBatch& b);
hipError_t run_kv_attention(const KvAttnArgs& a, hipStream_t st);

// The attention kernel of one code width and head size (a translation unit of its own).
template <int BITS, int D>
hipError_t run_kv_attention_form(const KvAttnArgs& a, hipStream_t st);

// 16-row tiles of a wave where each wave has its own rows: what 256 registers hold.
constexpr int kv_many_tiles(int head_dim) { return head_dim == 256 ? 1 : 2; }
constexpr int kv_many_waves(int head_dim) { return head_dim == 64 ? 4 : 8; }
KvPlan kv_attention_plan(const KvCache& c, const KvBatch& b, int heads_per_kv, int causal, int window, int sinks);
// Threads of a block.
inline int kv_plan_threads(const KvPlan& p) { return 64 * (p.row_waves == 1 ? p.key_waves : p.row_waves); }
// Rows of one (sequence, K/V head) in the partial results.
int64_t kv_plan_rows(const KvPlan& p);

}  // namespace echo
