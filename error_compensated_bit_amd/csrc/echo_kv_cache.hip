// echo_kv_cache.hip -- rows of keys and values into a paged cache of 4- or
// 8-bit codes, and back.
//
// Both kernels stream: per row of D elements 2 D bytes of 16-bit values on one
// side and D * bits / 8 codes + 4 D / group bytes of parameters on the other.
// A lane has 8 consecutive elements (one 16-byte access), a row is an aligned
// run of D/8 lanes, and a group's minimum and maximum are a butterfly of DPP
// moves inside that run.  The order of the codes in a row is the attention
// kernel's (echo_kv_device.h): for keys a permutation of the lanes' words, for
// values a transposition of codes between lanes, three exchanges by DPP.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "echo_kv_device.h"
#include "echo_kv_internal.h"

namespace echo {
namespace kv {

constexpr int kThreads = kKvCacheThreads;

// One step of a minimum and a maximum between lanes.  Written out because the
// compiler keeps the move between lanes apart from the minimum and quiets its
// result first: 9 instructions a step in place of 3 (a lane exchange reads what
// the vector unit wrote two cycles before at the latest, hence the s_nop).
#define ECHO_KV_MINMAX(LANES)                                       \
  asm volatile("s_nop 1\n"                                          \
               "v_min_f32_dpp %0, %0, %0 " LANES " row_mask:0xf bank_mask:0xf bound_ctrl:0\n" \
               "v_max_f32_dpp %1, %1, %1 " LANES " row_mask:0xf bank_mask:0xf bound_ctrl:0"   \
               : "+v"(mn), "+v"(mx))

// Minimum and maximum over aligned runs of LANES = 4, 8 or 16 lanes.
template <int LANES>
__device__ __forceinline__ void run_minmax(float& mn, float& mx) {
  ECHO_KV_MINMAX("quad_perm:[1,0,3,2]");
  ECHO_KV_MINMAX("quad_perm:[2,3,0,1]");
  if constexpr (LANES >= 8) ECHO_KV_MINMAX("row_half_mirror");   // lane i <-> 7-i within 8
  if constexpr (LANES >= 16) ECHO_KV_MINMAX("row_mirror");       // lane i <-> 15-i within 16
}
#undef ECHO_KV_MINMAX

template <int DT>
__device__ __forceinline__ void load8(const void* p, int64_t e, u32x4 (&w)[DT == kKvF32 ? 2 : 1]) {
  const u32x4* q = reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(p) + e * (DT == kKvF32 ? 4 : 2));
  w[0] = __builtin_nontemporal_load(q);
  if constexpr (DT == kKvF32) w[1] = __builtin_nontemporal_load(q + 1);
}
template <int DT>
__device__ __forceinline__ void widen8(const u32x4 (&w)[DT == kKvF32 ? 2 : 1], float* v) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (DT == kKvF32) v[i] = __uint_as_float(w[i / 4][i % 4]);
    else if constexpr (DT == kKvF16) v[i] = f16_to_f32(i & 1 ? w[0][i / 2] >> 16 : w[0][i / 2] & 0xffffu);
    else v[i] = (float)__builtin_bit_cast(__bf16, (uint16_t)(i & 1 ? w[0][i / 2] >> 16 : w[0][i / 2] & 0xffffu));
  }
}

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

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
    for (int i = 0; i < 4; ++i) {
      const f32x2 two = {v[2 * i], v[2 * i + 1]};
      if constexpr (DT == kKvF16) w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(two, f16x2));
      else w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(two, bf16x2));
    }
    __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + e));
  }
}

struct QParams {
  float zf, sf, inv;
  uint32_t word;  // step bits | zero bits << 16
};

// Group parameters: the all-reduce quantizer's, without the compiler's full
// divisions, which cost a fifth of the kernel's instructions.  span / qmax
// is the product with the rounded reciprocal and one correction, which rounds
// correctly wherever the quotient does not vanish in fp16 (below 2^-25 it is 0
// either way); spans beyond 65504 qmax give 65504.  1 / step is the hardware's
// reciprocal and one correction; it is right for every fp16 step.
template <int BITS>
__device__ __forceinline__ QParams group_params(float mn, float mx) {
  constexpr float qmax = (float)((1 << BITS) - 1);
  constexpr float rq = 1.0f / qmax;
  const float zc = fminf(fmaxf(mn, -65504.0f), 65504.0f);
  uint32_t zb = f32_to_f16(zc);
  zb = (zb == 0x8000u) ? 0u : zb;
  const float zf = f16_to_f32(zb);
  float span = mx - zf;
  span = span > 0.0f ? fminf(span, 65504.0f * qmax) : 0.0f;
  const float s0 = span * rq;
  const float s = fminf(fmaf(fmaf(-qmax, s0, span), rq, s0), 65504.0f);
  const uint32_t sb = f32_to_f16(s);
  const float sf = f16_to_f32(sb);
  const float y = __builtin_amdgcn_rcpf(sf);
  const float inv = sb ? fmaf(fmaf(-sf, y, 1.0f), y, y) : 0.0f;
  return QParams{zf, sf, inv, sb | (zb << 16)};
}

// Codes of 8 elements: w[0] of 8 nibbles, or w[0], w[1] of 4 bytes, in order.
template <int BITS>
__device__ __forceinline__ void encode8(const float* x, const QParams& q, uint32_t* w) {
  constexpr float qmax = (float)((1 << BITS) - 1);
  uint32_t b[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = __builtin_amdgcn_fmed3f((x[i] - q.zf) * q.inv, 0.0f, qmax);   // NaN: 0
    // the conversion rounds half to even
    b[i / 4] = __builtin_amdgcn_cvt_pk_u8_f32(t, i % 4, b[i / 4]);
  }
  if constexpr (BITS == 8) {
    w[0] = b[0];
    w[1] = b[1];
  } else {
    w[0] = __builtin_amdgcn_perm(b[1] | b[1] >> 4, b[0] | b[0] >> 4, 0x06040200u);
  }
}

template <int BITS>
__device__ __forceinline__ void decode8(const uint32_t* w, uint32_t word, float* x) {
  const float sf = f16_to_f32(word & 0xffffu), zf = f16_to_f32(word >> 16);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t c;
    if constexpr (BITS == 8) c = w[i / 4] >> (8 * (i % 4)) & 255u;
    else c = (i & 1 ? w[0] >> 4 & 0x0f0f0f0fu : w[0] & 0x0f0f0f0fu) >> (8 * (i / 2)) & 255u;
    x[i] = fmaf((float)c, sf, zf);
  }
}

// The transposition between a lane's 8 consecutive elements and the stored
// order of values, its own inverse.  Lane r of a row has the elements 8 r + j;
// with r = 2 i + p and the element's tile i and column m = 8 p + j, stored
// shares run over i at fixed m.  Exchanging bit b of i (lane bit b + 1) with bit
// b of j for b = 0, 1, 2 leaves lane (i, p) with the codes of column 8 p + i
// (D = 128; D = 256 keeps its highest bit of i in the lane; D = 64 has two bits
// to exchange, and j's third tells the lane's two half shares).
template <int BIT>
__device__ __forceinline__ uint32_t lane_xor(uint32_t v) {   // from lane ^ 2, 4 or 8
  if constexpr (BIT == 0) return __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xF, 0xF, true);   // quad_perm [2,3,0,1]
  if constexpr (BIT == 1)   // xor 7, then xor 3
    return __builtin_amdgcn_update_dpp(0, __builtin_amdgcn_update_dpp(0, v, 0x141, 0xF, 0xF, true), 0x1B, 0xF, 0xF, true);
  return __builtin_amdgcn_update_dpp(0, v, 0x128, 0xF, 0xF, true);                          // row_ror:8
}
template <int BITS, int BIT>
__device__ __forceinline__ void exchange_bit(uint32_t* w) {
  const bool up = threadIdx.x >> (BIT + 1) & 1u;
  constexpr int kDist = BITS << BIT;   // distance of the exchanged codes in bits
  if constexpr (kDist == 32) {
    const uint32_t got = lane_xor<BIT>(up ? w[0] : w[1]);
    if (up) w[0] = got;
    else w[1] = got;
  } else {
    constexpr uint32_t kLow = kDist == 4 ? 0x0f0f0f0fu : kDist == 8 ? 0x00ff00ffu : 0x0000ffffu;
    const uint32_t keep = up ? ~kLow : kLow, turn = up ? kDist : 32 - kDist;
#pragma unroll
    for (int i = 0; i < BITS / 4; ++i) {
      const uint32_t got = lane_xor<BIT>(w[i]);
      w[i] = (w[i] & keep) | (__builtin_amdgcn_alignbit(got, got, turn) & ~keep);
    }
  }
}
template <int BITS, int D>
__device__ __forceinline__ void transpose_values(uint32_t* w) {
  exchange_bit<BITS, 0>(w);
  exchange_bit<BITS, 1>(w);
  if constexpr (D >= 128) exchange_bit<BITS, 2>(w);
}

// Byte offset in a stored row of values of what lane `run` holds behind the
// transposition; D = 64: of its first half share, the second kHalf bytes on.
template <int BITS, int D>
__device__ __forceinline__ int value_place(int run) {
  constexpr int kUnit = D / 16 * BITS / 8;   // bytes of a column
  const int p = run & 1, i = run >> 1;
  if constexpr (D == 64) return (8 * p + i) * kUnit;
  else if constexpr (D == 128) return (8 * p + i) * kUnit;
  else return (8 * p + i % 8) * kUnit + i / 8 * (kUnit / 2);
}
template <int BITS, int D>
__device__ __forceinline__ void store_codes(uint8_t* row, int place, bool values, const uint32_t* w) {
  if constexpr (D == 64) {
    if (values) {
      constexpr int kHalf = 4 * (D / 16 * BITS / 8);   // column m + 4
      if constexpr (BITS == 4) {
        *reinterpret_cast<uint16_t*>(row + place) = (uint16_t)w[0];
        *reinterpret_cast<uint16_t*>(row + place + kHalf) = (uint16_t)(w[0] >> 16);
      } else {
        *reinterpret_cast<uint32_t*>(row + place) = w[0];
        *reinterpret_cast<uint32_t*>(row + place + kHalf) = w[1];
      }
      return;
    }
  }
  if constexpr (BITS == 4) *reinterpret_cast<uint32_t*>(row + place) = w[0];
  else *reinterpret_cast<u32x2*>(row + place) = u32x2{w[0], w[1]};
}
template <int BITS, int D>
__device__ __forceinline__ void load_codes(const uint8_t* row, int place, bool values, uint32_t* w) {
  if constexpr (D == 64) {
    if (values) {
      constexpr int kHalf = 4 * (D / 16 * BITS / 8);
      if constexpr (BITS == 4) {
        w[0] = *reinterpret_cast<const uint16_t*>(row + place) |
               (uint32_t)*reinterpret_cast<const uint16_t*>(row + place + kHalf) << 16;
      } else {
        w[0] = *reinterpret_cast<const uint32_t*>(row + place);
        w[1] = *reinterpret_cast<const uint32_t*>(row + place + kHalf);
      }
      return;
    }
  }
  if constexpr (BITS == 4) {
    w[0] = *reinterpret_cast<const uint32_t*>(row + place);
  } else {
    const u32x2 v = *reinterpret_cast<const u32x2*>(row + place);
    w[0] = v.x;
    w[1] = v.y;
  }
}

// Position of the 8-element run r in a stored row of keys, in runs.
template <int D>
__device__ __forceinline__ int key_run(int r) {
  return (r % 4) * (D / 32) + r / 4;
}

constexpr int kMaxTokens = 256;   // of a block

// A block's tokens t0 .. t0 + count - 1: for each, its row of head 0 in the
// cache, -1 where it has no place.  A wave looks up 64 tokens, mostly of one
// sequence; where they are not, each lane finds its own by bisection.  Looking
// places up once per token and block keeps the chain of dependent loads out of
// the rows' way.
__device__ __forceinline__ void look_up(const KvCache& c, const KvBatch& b, int t0, int count, int64_t* place) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  if (wave * 64 >= count) return;
  const int first = t0 + wave * 64, last = min(first + 63, t0 + count - 1);
  const int t = min(first + (int)(threadIdx.x % 64), last);
  SeqEntry s = seq_of_row(b, first);
  if (s.seq < 0 || last >= s.end) {
    int lo = s.seq < 0 ? 0 : s.seq, hi = seq_of_row(b, last).seq;
    const bool any = hi >= 0;
    while (lo < hi) {
      const int mid = lo + (hi - lo + 1) / 2;
      if (b.row_start[mid] <= t) lo = mid;
      else hi = mid - 1;
    }
    if (any) s = SeqEntry{lo, b.row_start[lo], b.row_start[lo + 1], b.kv_len[lo]};
  }
  place[wave * 64 + threadIdx.x % 64] = row_place(c, b, s, t);
}

// Rows (token, head) of a block, head-major: neighbouring rows are neighbours in
// the cache, whose short rows share lines.  Lane `run` of D/8 lanes has 8
// consecutive elements of a row; a pass covers kRows rows of the block's
// `tokens` * heads, and token, head and offset move from pass to pass by
// additions.
template <int D>
struct Rows {
  static constexpr int kLanes = D / 8;
  static constexpr int kRows = kThreads / kLanes;
  int t, h;            // token of the block, head
  int64_t e;           // element offset of the lane's elements from the block's first row
  __device__ __forceinline__ Rows(const KvRows& x, int tokens) {
    const int row = threadIdx.x / kLanes;
    h = row / tokens;
    t = row - h * tokens;
    e = (int64_t)t * x.row_stride + (int64_t)h * x.head_stride + threadIdx.x % kLanes * 8;
  }
  __device__ __forceinline__ void next(const KvRows& x, int tokens) {
    const int dh = kRows / tokens, dt = kRows - dh * tokens;
    t += dt;
    h += dh;
    e += (int64_t)dt * x.row_stride + (int64_t)dh * x.head_stride;
    if (t >= tokens) {
      t -= tokens;
      h += 1;
      e += x.head_stride - (int64_t)tokens * x.row_stride;
    }
  }
};

// grid.x: blocks of `tokens` tokens; grid.y: 0 keys, 1 values.  U passes' loads
// are in flight together.
template <int BITS, int D, int G, int DT, int U>
__global__ __launch_bounds__(kThreads) void k_kv_write(KvCache c, KvBatch b, KvRows k, KvRows v, int tokens) {
  using R = Rows<D>;
  __shared__ int64_t place[kMaxTokens];
  const bool values = blockIdx.y == 1;
  const KvRows& in = values ? v : k;
  uint8_t* const out_codes = values ? c.v_codes : c.k_codes;
  uint32_t* const out_params = values ? c.v_params : c.k_params;
  const int t0 = blockIdx.x * tokens, count = min(tokens, b.rows - t0);
  const void* from = static_cast<const uint8_t*>(in.p) + (int64_t)t0 * in.row_stride * (DT == kKvF32 ? 4 : 2);
  const int run = threadIdx.x % R::kLanes;
  const int at_codes = values ? value_place<BITS, D>(run) : key_run<D>(run) * BITS;
  R load(in, tokens), store = load;
  bool looked_up = false;
  for (int r0 = 0; r0 < tokens * c.kv_heads; r0 += U * R::kRows) {
    u32x4 raw[U][DT == kKvF32 ? 2 : 1];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (u32x4& w : raw[u]) w = u32x4{0, 0, 0, 0};
      if (load.t < count && load.h < c.kv_heads) load8<DT>(from, load.e, raw[u]);
      load.next(in, tokens);
    }
    if (!looked_up) {   // behind the first loads
      look_up(c, b, t0, count, place);
      __syncthreads();
      looked_up = true;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float x[8];
      widen8<DT>(raw[u], x);
      float mn = x[0], mx = x[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) {
        mn = fminf(mn, x[i]);
        mx = fmaxf(mx, x[i]);
      }
      run_minmax<G / 8>(mn, mx);
      const QParams q = group_params<BITS>(mn, mx);
      uint32_t w[BITS / 4];
      encode8<BITS>(x, q, w);
      if (values) transpose_values<BITS, D>(w);   // every lane of a row takes part
      const int64_t at0 = store.t < count && store.h < c.kv_heads ? place[store.t] : -1;
      if (at0 >= 0) {
        const int64_t at = at0 + ((int64_t)store.h << c.page_shift);
        store_codes<BITS, D>(out_codes + at * (D * BITS / 8), at_codes, values, w);
        if (run % (G / 8) == 0) out_params[at * (D / G) + run / (G / 8)] = q.word;
      }
      store.next(in, tokens);
    }
  }
}

template <int BITS, int D, int G, int DT, int U>
__global__ __launch_bounds__(kThreads) void k_kv_read(KvCache c, KvBatch b, KvRows k, KvRows v, int tokens) {
  using R = Rows<D>;
  __shared__ int64_t place[kMaxTokens];
  const bool values = blockIdx.y == 1;
  const KvRows& out = values ? v : k;
  const uint8_t* const in_codes = values ? c.v_codes : c.k_codes;
  const uint32_t* const in_params = values ? c.v_params : c.k_params;
  const int t0 = blockIdx.x * tokens, count = min(tokens, b.rows - t0);
  void* to = static_cast<uint8_t*>(out.p) + (int64_t)t0 * out.row_stride * (DT == kKvF32 ? 4 : 2);
  const int run = threadIdx.x % R::kLanes;
  const int at_codes = values ? value_place<BITS, D>(run) : key_run<D>(run) * BITS;
  R load(out, tokens), store = load;
  look_up(c, b, t0, count, place);
  __syncthreads();
  for (int r0 = 0; r0 < tokens * c.kv_heads; r0 += U * R::kRows) {
    uint32_t w[U][BITS / 4], word[U];
    bool there[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t at0 = load.t < count && load.h < c.kv_heads ? place[load.t] : -1;
      there[u] = at0 >= 0;
      word[u] = 0;
#pragma unroll
      for (uint32_t& i : w[u]) i = 0;
      if (there[u]) {
        const int64_t at = at0 + ((int64_t)load.h << c.page_shift);
        load_codes<BITS, D>(in_codes + at * (D * BITS / 8), at_codes, values, w[u]);
        word[u] = in_params[at * (D / G) + run / (G / 8)];
      }
      load.next(out, tokens);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (values) transpose_values<BITS, D>(w[u]);
      float x[8];
      decode8<BITS>(w[u], word[u], x);
      if (there[u]) store8<DT>(to, store.e, x);
      store.next(out, tokens);
    }
  }
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

// Tokens of a block: about 256 rows, fewer while that leaves compute units idle.
int block_tokens(const KvCache& c, const KvBatch& b) {
  int64_t tokens = 256 / c.kv_heads;
  const int64_t spread = ((int64_t)b.rows + 511) / 512;
  if (tokens > spread) tokens = spread;
  if (tokens > kv::kMaxTokens) tokens = kv::kMaxTokens;
  return (int)(tokens < 1 ? 1 : tokens);
}

constexpr int kPasses = 4;   // rows of a lane in flight together

}  // namespace

int64_t kv_cache_blocks(const KvCache& c, const KvBatch& b) {
  const int tokens = block_tokens(c, b);
  return ((int64_t)b.rows + tokens - 1) / tokens;
}

hipError_t run_kv_write(const KvWriteArgs& a, hipStream_t st) {
  const int tokens = block_tokens(a.c, a.b);
  return with_form(a.c, a.k.dtype, [&](auto B, auto D, auto G, auto T) {
    return kv_launch(kv::k_kv_write<B(), D(), G(), T(), kPasses>, dim3((unsigned)kv_cache_blocks(a.c, a.b), 2),
                     dim3(kv::kThreads), st, a.c, a.b, a.k, a.v, tokens);
  });
}

hipError_t run_kv_read(const KvWriteArgs& a, hipStream_t st) {
  const int tokens = block_tokens(a.c, a.b);
  return with_form(a.c, a.k.dtype, [&](auto B, auto D, auto G, auto T) {
    return kv_launch(kv::k_kv_read<B(), D(), G(), T(), kPasses>, dim3((unsigned)kv_cache_blocks(a.c, a.b), 2),
                     dim3(kv::kThreads), st, a.c, a.b, a.k, a.v, tokens);
  });
}

}  // namespace echo
