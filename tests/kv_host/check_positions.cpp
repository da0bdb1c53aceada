// Positions of the quantized K/V cache kernels on the host: attention puts a
// row where the write puts it, whatever the lengths and bounds, and the tiles
// of a block cover every key that rows at such positions see.
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "echo_kv_device.h"
#include "echo_kv_internal.h"

using namespace echo;

static std::mt19937 rng(2);
static int uniform(int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(rng); }
#define CHECK(c) \
  do { if (!(c)) { std::printf("line %d: %s\n", __LINE__, #c); std::exit(1); } } while (0)

static int any_length(int around) {
  const int k = uniform(0, 5);
  return k == 0 ? (int)rng() : k == 1 ? 0x7fffffff - uniform(0, 3) : k == 2 ? -0x7fffffff - 1 : uniform(-5, around);
}

static void as_written() {
  for (int trial = 0; trial < 20000; ++trial) {
    KvAttnArgs a{};
    a.b.seqs = 3;
    a.b.rows = uniform(1, 200);
    a.b.max_new = a.b.rows;
    a.b.max_len = uniform(0, 300);
    a.b.table_stride = uniform(1, 6);
    a.c.page_shift = uniform(4, 6);
    a.c.kv_heads = 1;
    a.c.num_pages = a.b.table_stride;
    std::vector<int32_t> table(3 * a.b.table_stride);
    for (size_t i = 0; i < table.size(); ++i) table[i] = (int32_t)(i % a.b.table_stride);
    int32_t start[4] = {uniform(-3, 5), 0, 0, 0}, len[3];
    for (int i = 0; i < 3; ++i) {
      start[i + 1] = start[i] + (uniform(0, 20) == 0 ? 0x7fffffff - 100000 * (i + 1) - std::max(start[i], 0) : uniform(0, 90));
      len[i] = any_length(400);
    }
    a.b.row_start = start;
    a.b.kv_len = len;
    a.b.page_table = table.data();
    for (int b = 0; b < 3; ++b) {
      if (start[b + 1] < start[b]) break;
      const kv::Seq s = kv::sequence(a, b);
      for (int i = 0; i < s.n; ++i) {
        const int64_t place = kv::row_place(a.c, a.b, kv::SeqEntry{b, start[b], start[b + 1], len[b]}, s.first + i);
        const int64_t pos = (int64_t)s.pos + i;
        CHECK(pos < 0x7fffffff && pos > -0x80000000ll);
        if (place >= 0) CHECK(place == pos && pos < s.len);
        else CHECK(pos < 0 || pos >= s.len);
      }
    }
  }
}

static bool visible(const KvAttnArgs& a, int64_t pos, int j) {
  if (!a.causal) return true;
  return j <= pos && (a.window == 0 || pos - j < a.window || j < a.sinks);
}

static void tiles() {
  for (int trial = 0; trial < 6000; ++trial) {
    KvAttnArgs a{};
    a.causal = uniform(0, 3) > 0;
    a.window = a.causal && uniform(0, 1) ? (uniform(0, 5) ? uniform(1, 700) : 0x7fffffff) : 0;
    a.sinks = a.window ? uniform(0, 1) * (uniform(0, 5) ? uniform(0, 200) : 0x7fffffff) : 0;
    a.heads_per_kv = uniform(1, 20);
    a.c.head_dim = 64 << uniform(0, 2);
    a.c.bits = uniform(0, 1) ? 4 : 8;
    a.c.kv_heads = uniform(1, 8);
    a.b.seqs = uniform(1, 40);
    a.b.max_len = uniform(0, 1) ? uniform(1, 400) : uniform(1, 20000);
    a.b.max_new = uniform(0, 1) ? uniform(1, 8) : uniform(1, 500);
    a.plan = kv_attention_plan(a.c, a.b, a.heads_per_kv, a.causal, a.window, a.sinks);
    const KvPlan& p = a.plan;
    const int block_rows = p.row_tiles * 16 * p.row_waves;
    const int len = uniform(0, a.b.max_len), n = uniform(1, a.b.max_new);
    // of all n rows, any number behind the keys or before the first position
    const int64_t pos = uniform(0, 4) ? (int64_t)len - n + uniform(-900, 900)
                                      : uniform(0, 1) ? 0x7ffffffell - n : -0x7fffffffll;
    const int rows = n * a.heads_per_kv, rb = uniform(0, (rows - 1) / block_rows);
    const int row0 = rb * block_rows, row1 = std::min(row0 + block_rows, rows) - 1;
    const kv::Span span = kv::key_span(a, len, len - pos, row0 / a.heads_per_kv, row1 / a.heads_per_kv);
    CHECK(span.tiles >= 0 && (int64_t)p.splits * p.split_tiles >= span.tiles);
    std::vector<char> covered(len + 1, 0);
    int before = -1;
    for (int t = 0; t < span.tiles; ++t) {
      const int tb = span.token(t);
      CHECK(tb % kv::kTile == 0 && tb > before && tb < len);
      before = tb;
      for (int j = tb; j < std::min(tb + kv::kTile, len); ++j) covered[j] = 1;
    }
    for (int i = row0 / a.heads_per_kv; i <= row1 / a.heads_per_kv; ++i)
      for (int j = 0; j < len; ++j)
        if (visible(a, pos + i, j)) CHECK(covered[j]);
  }
}

int main() {
  as_written();
  tiles();
  std::puts("ok");
  return 0;
}
