// echo_kv_device.h -- device helpers of the quantized K/V cache kernels.
//
// The quantizer is the all-reduce's: zero = fp16(min), step = fp16((max -
// zero) / qmax), code = round-half-even((x - zero) * (1 / step)), value =
// fma(code, step, zero), each operation in binary32 without contraction.
//
// Order of the codes inside a row of D elements.  The attention kernel feeds
// the 16x16x32 f16 matrix instruction straight from global memory, so each
// row is stored in the order in which a wave's lanes take it:
//   keys: lane group `quad` (of 4) holds, for every 32-element slice w, the 8
//     elements 32 w + 8 quad + 0..7.  Its D/4 codes are contiguous: the row is
//     the 8-element runs in the order quad-major, w-minor.
//   values: lane m (of 16) holds the elements 16 i + m of every 16-element
//     tile i; its D/16 codes are contiguous.
// 4-bit codes: the earlier code in the low nibble.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "echo_kv_internal.h"

namespace echo {
namespace kv {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float bf16_to_f32(uint32_t b) { return __uint_as_float(b << 16); }
__device__ __forceinline__ float f16_to_f32(uint32_t h) {
  return (float)__builtin_bit_cast(_Float16, (uint16_t)h);
}
__device__ __forceinline__ uint32_t f32_to_f16(float f) {
  return __builtin_bit_cast(uint16_t, (_Float16)f);
}
__device__ __forceinline__ uint32_t f32_to_bf16(float f) {
  return __builtin_bit_cast(uint16_t, (__bf16)f);
}

struct QParams {
  float zf, sf, inv;
  uint32_t word;  // step bits | zero bits << 16
};

template <int BITS>
__device__ __forceinline__ QParams group_params(float mn, float mx) {
  constexpr float qmax = (float)((1 << BITS) - 1);
  const float zc = fminf(fmaxf(mn, -65504.0f), 65504.0f);
  uint32_t zb = f32_to_f16(zc);
  zb = (zb == 0x8000u) ? 0u : zb;
  const float zf = f16_to_f32(zb);
  float s = (mx - zf) / qmax;
  s = (s > 0.0f) ? fminf(s, 65504.0f) : 0.0f;
  const uint32_t sb = f32_to_f16(s);
  const float sf = f16_to_f32(sb);
  const float inv = (sf > 0.0f) ? 1.0f / sf : 0.0f;
  return QParams{zf, sf, inv, sb | (zb << 16)};
}

template <int BITS>
__device__ __forceinline__ uint32_t encode(float v, const QParams& q) {
  constexpr float qmax = (float)((1 << BITS) - 1);
  const float t = (v - q.zf) * q.inv;
  return (uint32_t)fminf(fmaxf(rintf(t), 0.0f), qmax);
}

// Largest b in [0, seqs) with row_start[b] <= t, -1 if there is none; t is the
// same in all lanes, and 64 candidates are looked at per step, so that up to
// 64 sequences cost one load.  Ends for any contents of row_start.
__device__ __forceinline__ int seq_of_row(const int32_t* __restrict__ row_start, int seqs, int t) {
  const int lane = threadIdx.x % 64;
  int lo = 0, hi = seqs;
  for (;;) {
    const int stride = (hi - lo + 63) / 64;
    const int64_t i = (int64_t)lo + (int64_t)lane * stride;
    const bool le = i < hi && row_start[i] <= t;
    const int c = __popcll(__ballot(le));
    if (c == 0) return lo > 0 ? lo : -1;
    lo += (c - 1) * stride;
    if (stride == 1) return lo;
    hi = lo + stride < hi ? lo + stride : hi;
  }
}

// Slot of row t of the packed arrays in one head's plane of a page, or
// page < 0 where the row has none: rows outside every sequence, positions
// outside the page table, entries that name no page.
struct RowSlot {
  int64_t page;
  int32_t slot;
};
__device__ __forceinline__ RowSlot row_slot(const KvCache& c, const KvBatch& b, int seq, int t) {
  RowSlot r{-1, 0};
  if (seq < 0 || t < b.row_start[seq]) return r;
  const int end = b.row_start[seq + 1];
  if (t >= end) return r;
  const int64_t pos = (int64_t)b.kv_len[seq] - end + t;
  if (pos < 0 || pos >= b.max_len) return r;
  const int64_t pi = pos >> c.page_shift;
  if (pi >= b.table_stride) return r;
  const int64_t page = b.page_table[(int64_t)seq * b.table_stride + pi];
  if (page < 0 || page >= c.num_pages) return r;
  r.page = page;
  r.slot = (int)(pos & ((1 << c.page_shift) - 1));
  return r;
}

// ---- shared by the attention kernel and the one that joins its splits
constexpr int kTile = 32;            // keys per step
constexpr int kWaves = 4;            // waves per block
constexpr float kLowest = -3.0e38f;  // running maximum before any key: below every finite score

// The keys a block's rows can see, as tiles: those below `t1` start at 0, the
// others at `start`; a window skips what lies between the first keys (sinks)
// and the earliest row's window.
struct Span {
  int t1, start, tiles;
  __device__ __forceinline__ int token(int t) const { return t < t1 ? t * kTile : start + (t - t1) * kTile; }
};

// What the rows of tokens i0 .. i1 (of n new ones) see of a sequence of `len` keys.
__device__ __forceinline__ Span key_span(const KvAttnArgs& a, int len, int n, int i0, int i1) {
  Span s{0, 0, 0};
  int end = len;
  if (a.causal) {
    end = len - n + i1 + 1;
    end = end < len ? end : len;
  }
  if (end <= 0) return s;
  if (a.window > 0) {
    const int64_t lo = (int64_t)len - n + i0 - a.window + 1;
    const int first = lo > 0 ? (int)lo / kTile * kTile : 0;
    const int sinks = a.sinks < end ? a.sinks : end;
    const int s_end = (sinks + kTile - 1) / kTile * kTile;
    if (s_end < first) {
      s.t1 = s_end / kTile;
      s.start = first;
    }
  }
  s.tiles = s.t1 + (end - s.start + kTile - 1) / kTile;
  return s;
}

// One sequence's rows: the first one's index in the packed arrays, how many it
// has, how many of them the call computes, and its keys.  Any contents of the
// device arrays give ranges inside the caller's bounds.
struct Seq {
  int first, n, computed, len;
};
__device__ __forceinline__ Seq sequence(const KvAttnArgs& a, int b) {
  Seq s;
  int lo = a.b.row_start[b], hi = a.b.row_start[b + 1];
  lo = lo < 0 ? 0 : lo > a.b.rows ? a.b.rows : lo;
  hi = hi < lo ? lo : hi > a.b.rows ? a.b.rows : hi;
  s.first = lo;
  s.n = hi - lo;
  s.computed = s.n < a.b.max_new ? s.n : a.b.max_new;
  const int64_t room = a.b.table_stride << a.c.page_shift;
  int64_t len = a.b.kv_len[b];
  len = len < 0 ? 0 : len > a.b.max_len ? a.b.max_len : len;
  s.len = (int)(len < room ? len : room);
  return s;
}

// One (m, l) pair and one output row of D floats of every split of a query row.
__device__ __forceinline__ int64_t part_index(const KvAttnArgs& a, int b, int hk, int prows, int row, int split) {
  return (((int64_t)b * a.c.kv_heads + hk) * prows + row) * a.plan.splits + split;
}

template <typename T>
struct Same {
  using type = T;
};

}  // namespace kv

// Launch with the launch's own status; no pending error of the caller's is read or cleared.
template <typename... Params>
hipError_t kv_launch(void (*kernel)(Params...), dim3 grid, dim3 block, hipStream_t st,
                     typename kv::Same<Params>::type... args) {
  void* ptrs[] = {static_cast<void*>(&args)...};
  return hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, block, ptrs, 0, st);
}

}  // namespace echo
