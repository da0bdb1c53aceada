// echo_kv_plan.hip -- how an attention call is cut into blocks, and the choice
// of the kernel's form.  Both depend on the call's sizes only, so that a
// workspace can be sized, and a captured call replayed, whatever the lengths in
// device memory are.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "echo_kv_internal.h"

namespace echo {

// Rows one block covers under a plan.
static int plan_block_rows(const KvPlan& p) { return p.row_tiles * 16 * p.row_waves; }

int64_t kv_plan_rows(const KvPlan& p) { return (int64_t)p.row_blocks * plan_block_rows(p); }

KvPlan kv_attention_plan(const KvCache& c, const KvBatch& b, int heads_per_kv, int causal, int window, int sinks) {
  KvPlan p;
  const int64_t rows = (int64_t)b.max_new * heads_per_kv;
  const int64_t pairs = (int64_t)b.seqs * c.kv_heads;
  const bool thin = pairs <= 128;   // fewer than half the compute units: another block of rows costs nothing
  // Few rows: the waves of a block share them and take turns over the keys; each
  // further block of rows unpacks all codes again.  Many: each wave has its own
  // rows and the codes are unpacked once.  Measured, 3000-4096 keys a sequence,
  // us (few / many): 128 elements, 512 pairs, 32 rows 47 / 250, 128 rows 164 / 258,
  // 256 rows 316 / 273; 256 elements, 512 pairs, 40 rows 224 / 257, 128 rows
  // 594 / 284, 128 pairs, 128 rows 131 / 155; 64 elements, 512 pairs, 128 rows
  // 108 / 127, 192 rows 156 / 223.
  const int64_t few = c.head_dim == 256 && !thin ? 48 : 128;
  p.key_waves = 4;
  if (rows <= few) {
    p.row_waves = 1;
    // two tiles of rows a wave share the unpacking, one gives twice the blocks
    // and half the rows to join: 24 rows, 512 pairs 70 / 49 us (one / two), 128
    // pairs 26 / 30 us, 8 pairs of 32768 keys 36 / 64 us; with 256 elements two
    // do not fit the registers of two waves a SIMD
    p.row_tiles = rows <= 16 || c.head_dim == 256 || (rows <= 32 && thin) ? 1 : 2;
  } else {
    p.row_waves = kv_many_waves(c.head_dim);
    p.row_tiles = kv_many_tiles(c.head_dim);
  }
  const int64_t block_rows = plan_block_rows(p);
  p.row_blocks = (int32_t)((rows + block_rows - 1) / block_rows);
  int64_t span = b.max_len;
  if (causal && window > 0) {
    const int64_t seen = (int64_t)window + block_rows / heads_per_kv + 1 + sinks + 4 * 32;   // and the tiles that are cut
    span = seen < span ? seen : span;
  }
  const int64_t tiles = (span + 31) / 32 > 0 ? (span + 31) / 32 : 1;
  const int64_t blocks = pairs * p.row_blocks;
  // Keys are split until there is a block for every compute unit, not into fewer
  // than 16 tiles: more and shorter blocks pay their start, their end and the
  // join more often (4 sequences of 131072 keys: 105 us with 256 blocks, 108 with
  // 512, 125 with 1536; one of 512 keys: 8.3 us whole, 9.7 in two).
  int64_t splits = 256 / blocks;
  if (splits > tiles / 16) splits = tiles / 16;
  // One block joins the parts of its rows: about 2 us for every split and 4096
  // elements where each wave has its own rows, a quarter of that where they share
  // them, against 1.2 and 0.15 us for a tile of keys.  The sum is least where
  // splits^2 * passes = tiles * 0.6 (0.3); us without / with this bound: 256 rows
  // after 16384 keys 493 / 218, 400 rows after 131072 keys 1852 / 533, 100 rows
  // after 32768 keys 130 / 57, one row after 131072 keys 62 / 28.
  const int64_t passes = (block_rows * c.head_dim / 8 + 511) / 512;
  while (splits > 1 && splits * splits * passes * 10 > tiles * (p.row_waves == 1 ? 3 : 6)) --splits;
  if (splits < 1 || blocks > kKvCounters) splits = 1;
  const int64_t per = (tiles + splits - 1) / splits;
  // With a block or less for a compute unit, 8 waves a block take half the steps
  // (8 / 4 waves: one sequence of 32768 keys, 4 rows, 23 / 27 us; 128 pairs, 6143
  // keys, 40 rows, 8 bits, 56 / 70 us); 256 elements of 8 bits do not fit the
  // registers of two waves a SIMD.
  if (p.row_waves == 1 && blocks * splits <= 256 && c.bits * c.head_dim <= 1024) p.key_waves = 8;
  p.split_tiles = (int32_t)per;
  p.splits = (int32_t)((tiles + per - 1) / per);
  return p;
}

hipError_t run_kv_attention(const KvAttnArgs& a, hipStream_t st) {
  const int D = a.c.head_dim;
  if (a.c.bits == 4)
    return D == 64 ? run_kv_attention_form<4, 64>(a, st)
         : D == 128 ? run_kv_attention_form<4, 128>(a, st) : run_kv_attention_form<4, 256>(a, st);
  return D == 64 ? run_kv_attention_form<8, 64>(a, st)
       : D == 128 ? run_kv_attention_form<8, 128>(a, st) : run_kv_attention_form<8, 256>(a, st);
}

}  // namespace echo
