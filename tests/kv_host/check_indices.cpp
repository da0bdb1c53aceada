// The index arithmetic of the quantized K/V cache kernels on the host: rows and
// places of arbitrary index arrays stay inside their bounds, and the tiles of a
// call's blocks cover every key a row sees, for random calls.
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "echo_kv_device.h"
#include "echo_kv_internal.h"

using namespace echo;

static std::mt19937 rng(1);
static int uniform(int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(rng); }
static int wide() {   // any int, small ones more often
  const int k = uniform(0, 3);
  return k == 0 ? (int)rng() : k == 1 ? uniform(-5, 5) : uniform(-200, 400);
}
#define CHECK(c) \
  do { if (!(c)) { std::printf("line %d: %s\n", __LINE__, #c); std::exit(1); } } while (0)

static void places() {
  for (int trial = 0; trial < 20000; ++trial) {
    KvCache c{};
    c.num_pages = uniform(1, 9);
    c.kv_heads = uniform(1, 5);
    c.page_shift = uniform(4, 8);
    KvBatch b{};
    b.table_stride = uniform(0, 6);
    b.seqs = uniform(1, 4);
    b.rows = uniform(1, 300);
    b.max_len = uniform(0, 2000);
    std::vector<int32_t> table(b.seqs * b.table_stride + 1, 0), page_of(1);
    for (auto& t : table) t = wide();
    b.page_table = table.data();
    kv::SeqEntry s{uniform(-1, b.seqs - 1), wide(), wide(), wide()};
    const int64_t p = kv::row_place(c, b, s, uniform(0, b.rows - 1));
    const int64_t plane = (int64_t)1 << c.page_shift;
    CHECK(p == -1 || (p >= 0 && p / (plane * c.kv_heads) < c.num_pages && p / plane % c.kv_heads == 0));
  }
}

static void sequences() {
  for (int trial = 0; trial < 20000; ++trial) {
    KvAttnArgs a{};
    a.b.seqs = 2;
    a.b.rows = uniform(0, 300);
    a.b.max_new = uniform(0, 40);
    a.b.max_len = uniform(0, 2000);
    a.b.table_stride = uniform(0, 6);
    a.c.page_shift = uniform(4, 8);
    int32_t start[3] = {wide(), wide(), wide()}, len[2] = {wide(), wide()};
    a.b.row_start = start;
    a.b.kv_len = len;
    for (int b = 0; b < 2; ++b) {
      const kv::Seq s = kv::sequence(a, b);
      CHECK(s.first >= 0 && s.n >= 0 && s.first + s.n <= a.b.rows);
      CHECK(s.computed >= 0 && s.computed <= s.n && s.computed <= a.b.max_new);
      CHECK(s.len >= 0 && s.len <= a.b.max_len && s.len <= a.b.table_stride << a.c.page_shift);
    }
  }
}

static bool visible(const KvAttnArgs& a, int pos, int j, int len) {
  if (j >= len) return false;
  if (!a.causal) return true;
  return j <= pos && (a.window == 0 || (int64_t)pos - j < a.window || j < a.sinks);
}

static void tiles() {
  for (int trial = 0; trial < 6000; ++trial) {
    KvAttnArgs a{};
    a.causal = uniform(0, 3) > 0;
    a.window = a.causal && uniform(0, 1) ? uniform(1, 700) : 0;
    a.sinks = a.window ? uniform(0, 1) * uniform(0, 200) : 0;
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
    CHECK((int64_t)p.row_blocks * block_rows >= (int64_t)a.b.max_new * a.heads_per_kv);
    CHECK(p.splits >= 1 && p.split_tiles >= 1);
    CHECK(p.splits == 1 || (int64_t)a.b.seqs * a.c.kv_heads * p.row_blocks <= kKvCounters);
    // one sequence of any length up to max_len; rows may outnumber its keys
    const int len = uniform(0, 3) ? uniform(0, a.b.max_len) : a.b.max_len;
    const int n = uniform(1, a.b.max_new);
    const int rows = n * a.heads_per_kv;
    const int rb = uniform(0, (rows - 1) / block_rows);
    const int row0 = rb * block_rows, row1 = std::min(row0 + block_rows, rows) - 1;
    const kv::Span span = kv::key_span(a, len, n, row0 / a.heads_per_kv, row1 / a.heads_per_kv);
    CHECK((int64_t)p.splits * p.split_tiles >= span.tiles);
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
        if (visible(a, len - n + i, j, len)) CHECK(covered[j]);
  }
}

int main() {
  places();
  sequences();
  tiles();
  std::puts("ok");
  return 0;
}
