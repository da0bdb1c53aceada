// echo_kv_join.hip -- how an attention call is cut into blocks, and the kernel
// that joins the results of the blocks that had parts of the same rows' keys.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "echo_kv_device.h"
#include "echo_kv_internal.h"

namespace echo {
namespace kv {

// Join the splits of a query row: one wave per row, D/64 elements per lane.
// grid.x: 4 rows of all (K/V head, row) pairs, grid.y: sequence.
template <int D>
__global__ __launch_bounds__(kWaves * 64) void k_kv_join(KvAttnArgs a, int block_rows) {
  constexpr int E = D / 64;
  const int b = blockIdx.y, lane = threadIdx.x % 64;
  const int prows = a.plan.row_blocks * block_rows;
  const int unit = __builtin_amdgcn_readfirstlane(blockIdx.x * kWaves + threadIdx.x / 64);
  const int hk = unit / prows, row = unit - hk * prows;
  const Seq sq = sequence(a, b);
  const int rows = sq.computed * a.heads_per_kv;
  if (hk >= a.c.kv_heads || row >= rows) return;
  const int row0 = row / block_rows * block_rows, row1 = min(row0 + block_rows, rows) - 1;
  const Span span = key_span(a, sq.len, sq.n, row0 / a.heads_per_kv, row1 / a.heads_per_kv);
  const int active = (span.tiles + a.plan.split_tiles - 1) / a.plan.split_tiles;
  if (active <= 1) return;
  const int64_t at = part_index(a, b, hk, prows, row, 0);
  const float* ml = a.part_ml + at * 2;
  float top = kLowest;
  for (int s = lane; s < active; s += 64) top = fmaxf(top, ml[2 * s]);
#pragma unroll
  for (int x = 1; x < 64; x *= 2) top = fmaxf(top, __shfl_xor(top, x));
  float sum = 0.0f, o[E] = {};
#pragma unroll 4
  for (int s = 0; s < active; ++s) {
    const float f = __builtin_amdgcn_exp2f(ml[2 * s] - top);
    sum = fmaf(ml[2 * s + 1], f, sum);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(a.part_o[(at + s) * D + lane * E + e], f, o[e]);
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  const int i = row / a.heads_per_kv, h = hk * a.heads_per_kv + row - i * a.heads_per_kv;
  uint16_t* out = static_cast<uint16_t*>(a.out.p) + (int64_t)(sq.first + i) * a.out.row_stride +
                  (int64_t)h * a.out.head_stride + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) out[e] = (uint16_t)(a.out.dtype == kKvF16 ? f32_to_f16(o[e] * inv) : f32_to_bf16(o[e] * inv));
}

}  // namespace kv

// Rows one block covers under a plan.
static int plan_block_rows(const KvPlan& p) { return p.row_tiles * 16 * p.row_waves; }

int64_t kv_plan_rows(const KvPlan& p) { return (int64_t)p.row_blocks * plan_block_rows(p); }

KvPlan kv_attention_plan(const KvCache& c, const KvBatch& b, int heads_per_kv, int causal, int window, int sinks) {
  KvPlan p;
  const int64_t rows = (int64_t)b.max_new * heads_per_kv;
  const int most = c.head_dim == 256 ? 2 : 3;   // tiles of rows that several waves share
  p.key_waves = 4;
  if (rows <= 16 * most) {
    p.row_waves = 1;
    p.row_tiles = (int32_t)((rows + 15) / 16);
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
  const int64_t blocks = (int64_t)b.seqs * c.kv_heads * p.row_blocks;
  const int64_t target = 512, capt = 512, lst = 8;
  int64_t splits = target / blocks;
  const int64_t least = p.row_waves == 1 ? lst : 16;
  if (splits > tiles / least) splits = tiles / least;
  if (splits < 1) splits = 1;
  int64_t per = (tiles + splits - 1) / splits;
  if (p.row_waves == 1 && per > capt) per = capt;
  if (p.row_waves == 1 && p.row_tiles == 1 && blocks * splits <= 256) p.key_waves = 8;
  p.split_tiles = (int32_t)per;
  p.splits = (int32_t)((tiles + per - 1) / per);
  return p;
}

template <int D>
static hipError_t launch_join(const KvAttnArgs& a, hipStream_t st) {
  const int64_t units = (int64_t)a.c.kv_heads * kv_plan_rows(a.plan);
  return kv_launch(kv::k_kv_join<D>, dim3((unsigned)((units + kv::kWaves - 1) / kv::kWaves), a.b.seqs),
                   dim3(kv::kWaves * 64), st, a, plan_block_rows(a.plan));
}

hipError_t run_kv_attention(const KvAttnArgs& a, hipStream_t st) {
  const int D = a.c.head_dim;
  hipError_t e;
  if (a.c.bits == 4)
    e = D == 64 ? run_kv_attention_form<4, 64>(a, st)
      : D == 128 ? run_kv_attention_form<4, 128>(a, st) : run_kv_attention_form<4, 256>(a, st);
  else
    e = D == 64 ? run_kv_attention_form<8, 64>(a, st)
      : D == 128 ? run_kv_attention_form<8, 128>(a, st) : run_kv_attention_form<8, 256>(a, st);
  if (e != hipSuccess || a.plan.splits <= 1) return e;
  return D == 64 ? launch_join<64>(a, st) : D == 128 ? launch_join<128>(a, st) : launch_join<256>(a, st);
}

}  // namespace echo
