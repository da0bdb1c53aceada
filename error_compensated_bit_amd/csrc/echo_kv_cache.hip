// echo_kv_cache.hip -- rows of keys and values into a paged cache of 4- or
// 8-bit codes, and back.
//
// Both kernels stream: per row of D elements 2 D bytes of 16-bit values on one
// side and D * bits / 8 codes + 4 D / group bytes of parameters on the other.
// A lane has 8 consecutive elements (one 16-byte access), a row is an aligned
// run of D/8 lanes, and a group's minimum and maximum are a butterfly of DPP
// moves inside that run.  The order of the codes in a row is the attention
// kernel's (echo_kv_device.h): for keys that is a permutation of the lanes'
// words; for values the lanes exchange their codes through LDS.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "echo_kv_device.h"
#include "echo_kv_internal.h"

namespace echo {
namespace kv {

constexpr int kThreads = 256;

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}

// Minimum and maximum over aligned runs of LANES = 4, 8 or 16 lanes.
template <int LANES>
__device__ __forceinline__ void run_minmax(float& mn, float& mx) {
  mn = fminf(mn, dpp<0xB1>(mn));     // quad_perm [1,0,3,2]
  mx = fmaxf(mx, dpp<0xB1>(mx));
  mn = fminf(mn, dpp<0x4E>(mn));     // quad_perm [2,3,0,1]
  mx = fmaxf(mx, dpp<0x4E>(mx));
  if constexpr (LANES >= 8) {
    mn = fminf(mn, dpp<0x141>(mn));  // lane i <-> 7-i within 8
    mx = fmaxf(mx, dpp<0x141>(mx));
  }
  if constexpr (LANES >= 16) {
    mn = fminf(mn, dpp<0x140>(mn));  // lane i <-> 15-i within 16
    mx = fmaxf(mx, dpp<0x140>(mx));
  }
}

template <int DT>
__device__ __forceinline__ void load8(const void* p, int64_t e, float* v) {
  if constexpr (DT == kKvF32) {
    const f32x4* q = reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + e);
    const f32x4 a = __builtin_nontemporal_load(q), b = __builtin_nontemporal_load(q + 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
  } else {
    const u32x4 w = __builtin_nontemporal_load(
        reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + e));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = DT == kKvF16 ? f16_to_f32(w[i] & 0xffffu) : bf16_to_f32(w[i] & 0xffffu);
      v[2 * i + 1] = DT == kKvF16 ? f16_to_f32(w[i] >> 16) : bf16_to_f32(w[i] >> 16);
    }
  }
}

template <int DT>
__device__ __forceinline__ void store8(void* p, int64_t e, const float* v) {
  if constexpr (DT == kKvF32) {
    f32x4* q = reinterpret_cast<f32x4*>(static_cast<float*>(p) + e);
    const f32x4 a = {v[0], v[1], v[2], v[3]}, b = {v[4], v[5], v[6], v[7]};
    __builtin_nontemporal_store(a, q);
    __builtin_nontemporal_store(b, q + 1);
  } else {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = DT == kKvF16 ? f32_to_f16(v[2 * i]) | (f32_to_f16(v[2 * i + 1]) << 16)
                          : f32_to_bf16(v[2 * i]) | (f32_to_bf16(v[2 * i + 1]) << 16);
    __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + e));
  }
}

// Where a lane's 8 consecutive elements are and which slot they belong to.
// Rows are numbered token-major (token t, head h -> t * kv_heads + h).
template <int D>
struct Lane {
  static constexpr int kLanes = D / 8;                  // lanes per row
  static constexpr int kRows = kThreads / kLanes;       // rows per block
  int t, h, run;    // run: which 8 elements
};

template <int D>
__device__ __forceinline__ Lane<D> lane_of(int kv_heads) {
  Lane<D> l;
  l.run = threadIdx.x % Lane<D>::kLanes;
  const uint32_t row = blockIdx.x * (uint32_t)Lane<D>::kRows + threadIdx.x / Lane<D>::kLanes;   // below 2^31
  l.t = (int)(row / (uint32_t)kv_heads);
  l.h = (int)(row - (uint32_t)l.t * (uint32_t)kv_heads);
  return l;
}

// Sequence of this lane's token: found for the wave's first and last token
// together, and between the two by bisection.
template <int D>
__device__ __forceinline__ int lane_seq(const KvBatch& b, const Lane<D>& l) {
  const int t0 = __builtin_amdgcn_readfirstlane(l.t);
  const int t1 = __builtin_amdgcn_readlane(l.t, 63);
  int lo = seq_of_row(b.row_start, b.seqs, t0);
  if (t0 == t1) return lo;
  int hi = seq_of_row(b.row_start, b.seqs, t1);
  if (lo < 0) lo = 0;
  while (lo < hi) {
    const int mid = lo + (hi - lo + 1) / 2;
    if (b.row_start[mid] <= l.t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Element of position c in a stored row of values.
template <int D>
__device__ __forceinline__ int value_element(int c) {
  constexpr int kUnit = D / 16;
  return (c % kUnit) * 16 + c / kUnit;
}
// Position of the 8-element run r in a stored row of keys, in runs.
template <int D>
__device__ __forceinline__ int key_run(int r) {
  return (r % 4) * (D / 32) + r / 4;
}

// grid.y: 0 keys, 1 values.
template <int BITS, int D, int G, int DT>
__global__ __launch_bounds__(kThreads) void k_kv_write(KvCache c, KvBatch b, KvRows k, KvRows v) {
  using L = Lane<D>;
  __shared__ uint32_t exchange[kThreads * 2];
  const bool values = blockIdx.y == 1;
  const KvRows& in = values ? v : k;
  const L l = lane_of<D>(c.kv_heads);
  const bool exists = l.t < b.rows;
  const int seq = lane_seq<D>(b, l);
  RowSlot s{-1, 0};
  if (exists) s = row_slot(c, b, seq, l.t);
  float x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (exists)
    load8<DT>(in.p, (int64_t)l.t * in.row_stride + (int64_t)l.h * in.head_stride + l.run * 8, x);
  float mn = x[0], mx = x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    mn = fminf(mn, x[i]);
    mx = fmaxf(mx, x[i]);
  }
  run_minmax<G / 8>(mn, mx);
  const QParams q = group_params<BITS>(mn, mx);
  uint32_t code[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) code[i] = encode<BITS>(x[i], q);
  if (values) {   // whole blocks: every lane takes part in the exchange
    exchange[threadIdx.x * 2] = code[0] | code[1] << 8 | code[2] << 16 | code[3] << 24;
    exchange[threadIdx.x * 2 + 1] = code[4] | code[5] << 8 | code[6] << 16 | code[7] << 24;
    __syncthreads();
    const uint8_t* row = reinterpret_cast<const uint8_t*>(exchange) + threadIdx.x / L::kLanes * D;
#pragma unroll
    for (int i = 0; i < 8; ++i) code[i] = row[value_element<D>(l.run * 8 + i)];
  }
  if (s.page < 0) return;
  const int64_t r = ((s.page * c.kv_heads + l.h) << c.page_shift) + s.slot;
  uint8_t* codes = (values ? c.v_codes : c.k_codes) + r * (D * BITS / 8);
  const int at = values ? l.run : key_run<D>(l.run);
  if constexpr (BITS == 4) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) w |= code[i] << (4 * i);
    reinterpret_cast<uint32_t*>(codes)[at] = w;
  } else {
    const u32x2 w = {code[0] | code[1] << 8 | code[2] << 16 | code[3] << 24,
                     code[4] | code[5] << 8 | code[6] << 16 | code[7] << 24};
    reinterpret_cast<u32x2*>(codes)[at] = w;
  }
  if (l.run % (G / 8) == 0)
    (values ? c.v_params : c.k_params)[r * (D / G) + l.run / (G / 8)] = q.word;
}

template <int BITS, int D, int G, int DT>
__global__ __launch_bounds__(kThreads) void k_kv_read(KvCache c, KvBatch b, KvRows k, KvRows v) {
  using L = Lane<D>;
  const bool values = blockIdx.y == 1;
  const KvRows& out = values ? v : k;
  const L l = lane_of<D>(c.kv_heads);
  const int seq = lane_seq<D>(b, l);
  if (l.t >= b.rows) return;
  const RowSlot s = row_slot(c, b, seq, l.t);
  if (s.page < 0) return;
  const int64_t r = ((s.page * c.kv_heads + l.h) << c.page_shift) + s.slot;
  const uint8_t* codes = (values ? c.v_codes : c.k_codes) + r * (D * BITS / 8);
  const uint32_t word = (values ? c.v_params : c.k_params)[r * (D / G) + l.run / (G / 8)];
  uint32_t code[8];
  if (values) {
    // elements 8 run + i = tile run/2, column 8 (run % 2) + i: one code of each of 8 lanes' shares
    constexpr int kUnitBytes = D * BITS / 8 / 16;
    const int tile = l.run / 2, col = (l.run % 2) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t byte = codes[(col + i) * kUnitBytes + tile * BITS / 8];
      code[i] = BITS == 8 ? byte : (tile & 1 ? byte >> 4 : byte & 15u);
    }
  } else if constexpr (BITS == 4) {
    const uint32_t w = reinterpret_cast<const uint32_t*>(codes)[key_run<D>(l.run)];
#pragma unroll
    for (int i = 0; i < 8; ++i) code[i] = (w >> (4 * i)) & 15u;
  } else {
    const u32x2 w = reinterpret_cast<const u32x2*>(codes)[key_run<D>(l.run)];
#pragma unroll
    for (int i = 0; i < 8; ++i) code[i] = (w[i / 4] >> (8 * (i % 4))) & 255u;
  }
  const float sf = f16_to_f32(word & 0xffffu), zf = f16_to_f32(word >> 16);
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = fmaf((float)code[i], sf, zf);
  store8<DT>(out.p, (int64_t)l.t * out.row_stride + (int64_t)l.h * out.head_stride + l.run * 8, x);
}

}  // namespace kv

namespace {

template <int V>
using IC = std::integral_constant<int, V>;

template <typename F>
hipError_t with_form(const KvCache& c, int dtype, F&& f) {
  auto with_dtype = [&](auto B, auto D, auto G) {
    if (dtype == kKvBF16) return f(B, D, G, IC<kKvBF16>{});
    if (dtype == kKvF16) return f(B, D, G, IC<kKvF16>{});
    return f(B, D, G, IC<kKvF32>{});
  };
  auto with_group = [&](auto B, auto D) {
    if (c.group == 32) return with_dtype(B, D, IC<32>{});
    if (c.group == 64) return with_dtype(B, D, IC<64>{});
    if constexpr (D() >= 128) return with_dtype(B, D, IC<128>{});
    return hipErrorInvalidValue;   // refused before the launch
  };
  auto with_dim = [&](auto B) {
    if (c.head_dim == 64) return with_group(B, IC<64>{});
    if (c.head_dim == 128) return with_group(B, IC<128>{});
    return with_group(B, IC<256>{});
  };
  return c.bits == 4 ? with_dim(IC<4>{}) : with_dim(IC<8>{});
}

unsigned row_blocks(const KvWriteArgs& a) {
  const int64_t rows = (int64_t)a.b.rows * a.c.kv_heads, per = kv::kThreads / (a.c.head_dim / 8);
  return (unsigned)((rows + per - 1) / per);
}

}  // namespace

hipError_t run_kv_write(const KvWriteArgs& a, hipStream_t st) {
  return with_form(a.c, a.k.dtype, [&](auto B, auto D, auto G, auto T) {
    return kv_launch(kv::k_kv_write<B(), D(), G(), T()>, dim3(row_blocks(a), 2), dim3(kv::kThreads), st,
                     a.c, a.b, a.k, a.v);
  });
}

hipError_t run_kv_read(const KvWriteArgs& a, hipStream_t st) {
  return with_form(a.c, a.k.dtype, [&](auto B, auto D, auto G, auto T) {
    return kv_launch(kv::k_kv_read<B(), D(), G(), T()>, dim3(row_blocks(a), 2), dim3(kv::kThreads), st,
                     a.c, a.b, a.k, a.v);
  });
}

}  // namespace echo
