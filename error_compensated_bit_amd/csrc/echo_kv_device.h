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

// A sequence and its entries of the batch's arrays; seq < 0: none.
struct SeqEntry {
  int seq, start, end, len;
};

// The largest seq with row_start[seq] <= t; t is the same in all lanes, and 64
// candidates are looked at per step, in the last step with all their entries,
// so that up to 64 sequences cost one round of loads.  Ends for any contents.
__device__ __forceinline__ SeqEntry seq_of_row(const KvBatch& b, int t) {
  const int lane = threadIdx.x % 64;
  int lo = 0, hi = b.seqs;
  while (hi - lo > 64) {
    const int stride = (hi - lo + 63) / 64;
    const int64_t i = (int64_t)lo + (int64_t)lane * stride;
    const int c = __popcll(__ballot(i < hi && b.row_start[i] <= t));
    if (c == 0) break;
    lo += (c - 1) * stride;
    hi = lo + stride < hi ? lo + stride : hi;
  }
  int start = 0, end = 0, len = 0;
  const bool mine = lane < hi - lo;
  if (mine) {
    start = b.row_start[lo + lane];
    end = b.row_start[lo + lane + 1];
    len = b.kv_len[lo + lane];
  }
  const int c = __popcll(__ballot(mine && start <= t));
  const int at = c == 0 ? 0 : c - 1;
  return SeqEntry{c == 0 ? -1 : lo + at, __builtin_amdgcn_readlane(start, at), __builtin_amdgcn_readlane(end, at),
                  __builtin_amdgcn_readlane(len, at)};
}

// Row of head 0 in the cache that row t of the packed arrays belongs to, or -1
// where it has no place: rows outside every sequence, positions outside the
// page table, entries that name no page.
__host__ __device__ __forceinline__ int64_t row_place(const KvCache& c, const KvBatch& b, const SeqEntry& s, int t) {
  if (s.seq < 0 || t < s.start || t >= s.end) return -1;
  const int64_t pos = (int64_t)s.len - s.end + t;
  if (pos < 0 || pos >= b.max_len) return -1;
  const int64_t pi = pos >> c.page_shift;
  if (pi >= b.table_stride) return -1;
  const int64_t page = b.page_table[(int64_t)s.seq * b.table_stride + pi];
  if (page < 0 || page >= c.num_pages) return -1;
  return ((page * c.kv_heads) << c.page_shift) + (pos & ((1 << c.page_shift) - 1));
}

// ---- attention
constexpr int kTile = 32;            // keys per tile
constexpr float kLowest = -3.0e38f;  // running maximum before any key: below every finite score

// The keys a block's rows can see, as tiles: those below `t1` start at 0, the
// others at `start`; a window skips what lies between the first keys (sinks)
// and the earliest row's window.  The rows see no key from `end` on.
struct Span {
  int t1, start, tiles, end;
  __host__ __device__ __forceinline__ int token(int t) const { return t < t1 ? t * kTile : start + (t - t1) * kTile; }
};

// The first key that the window leaves to a row at position p; 32 bits hold it
// for any p and window.
__host__ __device__ __forceinline__ int window_start(int window, int p) {
  return window > 0 && p >= window ? p - window + 1 : 0;
}

// What the rows of tokens i0 .. i1 see of a sequence of `len` keys whose token 0
// sits at position len - n.
__host__ __device__ __forceinline__ Span key_span(const KvAttnArgs& a, int len, int64_t n, int i0, int i1) {
  Span s{0, 0, 0, 0};
  const int pos = (int)(len - n);
  int end = len;
  if (a.causal && pos + i1 < len) end = pos + i1 + 1;
  if (end <= 0) return s;
  s.end = end;
  if (a.window > 0) {
    int first = window_start(a.window, pos + i0);
    first = (first < len ? first : len) / kTile * kTile;   // rows behind the keys may see only the first ones
    const int sinks = a.sinks < end ? a.sinks : end;
    const int s_end = (sinks + kTile - 1) / kTile * kTile;
    if (s_end < first) {
      s.t1 = s_end / kTile;
      s.start = first;
    }
  }
  s.tiles = s.t1 + (end > s.start ? (end - s.start + kTile - 1) / kTile : 0);
  return s;
}

// One sequence's rows: the first one's index in the packed arrays and position,
// how many of them the call computes, and its keys.  The rows are the last
// positions of kv_len, as in row_place(), also where max_len or the page table
// leaves fewer keys.  Any contents of the device arrays give ranges inside the
// caller's bounds, and positions inside 32 bits: -2^31 < kv_len - row_end + row
// < 2^31 for rows below row_end.
struct Seq {
  int first, n, computed, len, pos;
};
__host__ __device__ __forceinline__ Seq sequence(const KvAttnArgs& a, int b) {
  Seq s;
  int lo = a.b.row_start[b];
  const int end = a.b.row_start[b + 1];
  int hi = end;
  lo = lo < 0 ? 0 : lo > a.b.rows ? a.b.rows : lo;
  hi = hi < lo ? lo : hi > a.b.rows ? a.b.rows : hi;
  s.first = lo;
  s.n = hi - lo;
  s.computed = s.n < a.b.max_new ? s.n : a.b.max_new;
  // in 32 bits: a 64-bit comparison would take its operands out of the scalar registers
  const int len = a.b.kv_len[b] < 0 ? 0 : a.b.kv_len[b];   // below 0 every position is, as with 0
  s.pos = s.n > 0 ? len - (end - lo) : 0;
  const int entries = (int)a.b.table_stride;   // at most 2^30
  const int room = entries > a.b.max_len >> a.c.page_shift ? a.b.max_len : entries << a.c.page_shift;
  s.len = len < room ? len : room;
  return s;
}

// One (m, l) pair and one output row of D floats of every split of a query row.
__host__ __device__ __forceinline__ int64_t part_index(const KvAttnArgs& a, int b, int hk, int prows, int row, int split) {
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
