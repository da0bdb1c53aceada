// echo_kv_attention.hip -- attention over a paged cache of 4- or 8-bit codes.
//
// Mathematics.  A cached key is k_j = s_jg c_j + z_jg inside group g (code c,
// step s, zero z), so a score is
//   q . k_j = sum_g s_jg (q . c_j)_g + z_jg Q_g,   Q_g = sum of q over group g,
// and with h half the code range (8 or 128) an output is
//   sum_j p_j v_j = sum_g [ sum_j (p_j s_jg) (c_j - h) + sum_j p_j (z_jg + h s_jg) ].
// Both matrix products then run on the codes themselves, which f16 holds
// exactly; nothing of the cache is rounded.  Moving h into the second sum
// keeps the two parts as small as the values, so that the f16 rounding of
// p_j s_jg (2^-12) counts relative to the values and not to the code range.
// Scores, maxima, sums and outputs are binary32.
//
// A code in the low bits of a half word IS a subnormal half, c 2^-24 (2^-20 for
// a 4-bit code one nibble higher): unpacking is one AND per two codes, and the
// powers of two come out of the fp32 result (and out of q for the higher
// nibbles).  The matrix instruction takes subnormal halves as they are.
//
// Layout.  Scores are computed transposed, S^T = K Q^T with 16 keys x 16 query
// rows per 16x16x32 instruction: its result gives lane (n = lane % 16, quad =
// lane / 16) the keys 4 quad + 0..3 of query row n, which is, for two such
// tiles, exactly the operand that O^T = V^T P^T wants from that lane.  So
// probabilities never leave their lane.  The cache stores keys and values in
// the order in which lanes take them (echo_kv_device.h).
//
// A wave works on NT tiles of 16 query rows (row = new token x query head of one
// K/V head) and walks the keys 32 or 64 at a time.  The running maximum moves
// only when a score exceeds it by more than 2^4, which keeps the rescaling of
// the output out of almost every step.  Two kernels: for few rows, where the
// cache's bytes bound the time, codes go from memory to registers; for many,
// where the arithmetic does, a block unpacks them once into LDS.  Where there
// are fewer blocks than compute units, the keys are split too and the last
// block to arrive joins the parts.
//
// Measured (bf16, 4 bits in groups of 128, 32 query and 8 K/V heads of 128
// elements): one new token of 4 sequences of about 126000 keys 106 us, 5.2 TB/s;
// of 64 sequences of 1100 to 4100 keys 45 us, 4.1 TB/s (the longest sequence's
// block is the whole time); 2048 new tokens after 16384 670 us, 872 TFLOP/s.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "echo_kv_device.h"
#include "echo_kv_internal.h"

namespace echo {
namespace kv {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

constexpr float kPeak = 10.0f;    // a probability of 1 at the running maximum enters the products as 2^10
constexpr float kSlack = 4.0f;    // log2 of how far a score may exceed the running maximum

__device__ __forceinline__ f32x4 mfma(f16x8 a, f16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f16x8 operand(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const u32x4 w = {a, b, c, d};
  return __builtin_bit_cast(f16x8, w);
}

// How the codes of 2 x 16 tokens lie in a wave's registers.
template <int BITS, int D, int G>
struct Tile {
  static constexpr int kRowBytes = D * BITS / 8;
  static constexpr int kKeyWords = kRowBytes / 16;       // words of a lane's share of one key row
  static constexpr int kUnitBytes = kRowBytes / 16;      // bytes of a lane's share of one value row
  static constexpr int kUnitWords = kUnitBytes < 4 ? 1 : kUnitBytes / 4;
  uint32_t k[2][kKeyWords];
  uint32_t v[2][4][kUnitWords];
};

template <int WORDS>
__device__ __forceinline__ void load_words(const uint8_t* __restrict__ p, uint32_t* w) {
  if constexpr (WORDS >= 4) {
#pragma unroll
    for (int i = 0; i < WORDS; i += 4) {
      const u32x4 a = *reinterpret_cast<const u32x4*>(p + 4 * i);
      w[i] = a.x, w[i + 1] = a.y, w[i + 2] = a.z, w[i + 3] = a.w;
    }
  } else if constexpr (WORDS == 2) {
    const u32x2 a = *reinterpret_cast<const u32x2*>(p);
    w[0] = a.x, w[1] = a.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

// Page of the 16 tokens at t, -1 where there is none; the same in all lanes, so
// it is a scalar load.
__device__ __forceinline__ int half_page(const KvCache& c, const int32_t* table, int len, int t) {
  typedef const int32_t __attribute__((address_space(4))) * scalar_ptr;
  int page = -1;
  if (t < len) page = ((scalar_ptr)(uintptr_t)table)[t >> c.page_shift];
  return page >= 0 && page < c.num_pages ? page : -1;
}
// The cache's row of token t in that page.  Without a page it is page 0, whose
// memory exists; what is read there is masked.
__device__ __forceinline__ int64_t half_row(const KvCache& c, int page, int hk, int t) {
  return (((int64_t)(page < 0 ? 0 : page) * c.kv_heads + hk) << c.page_shift) + (t & ((1 << c.page_shift) - 1));
}

// Pages of the two halves of the tile at token tb.
struct Pages {
  int p[2];
  __device__ __forceinline__ uint32_t ok() const { return (p[0] < 0 ? 0u : 1u) | (p[1] < 0 ? 0u : 2u); }
};
__device__ __forceinline__ Pages tile_pages(const KvCache& c, const int32_t* table, int len, int tb) {
  Pages r;
  r.p[0] = half_page(c, table, len, tb);
  // a tile lies in one page unless pages have 16 slots
  r.p[1] = c.page_shift == 4 ? half_page(c, table, len, tb + 16) : tb + 16 < len ? r.p[0] : -1;
  return r;
}
// The cache's rows of the two halves.
struct Halves {
  int64_t row[2];
};
__device__ __forceinline__ Halves tile_halves(const KvCache& c, const Pages& pages, int hk, int tb) {
  Halves h;
  h.row[0] = half_row(c, pages.p[0], hk, tb);
  h.row[1] = c.page_shift == 4 ? half_row(c, pages.p[1], hk, tb + 16) : h.row[0] + 16;
  return h;
}

template <int BITS, int D, int G>
__device__ __forceinline__ void load_tile(Tile<BITS, D, G>& x, const KvCache& c, const Halves& h) {
  using T = Tile<BITS, D, G>;
  const uint32_t n = threadIdx.x % 16, quad = threadIdx.x / 16 % 4;
  const uint32_t k_at = n * T::kRowBytes + quad * (T::kRowBytes / 4);
  const uint32_t v_at = quad * 4 * T::kRowBytes + n * T::kUnitBytes;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const uint8_t* kc = c.k_codes + h.row[s] * T::kRowBytes;
    const uint8_t* vc = c.v_codes + h.row[s] * T::kRowBytes;
    load_words<T::kKeyWords>(kc + k_at, x.k[s]);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if constexpr (T::kUnitBytes == 2) x.v[s][r][0] = *reinterpret_cast<const uint16_t*>(vc + v_at + r * T::kRowBytes);
      else load_words<T::kUnitWords>(vc + v_at + r * T::kRowBytes, x.v[s][r]);
    }
  }
}

// LDS written by other lanes of this wave is visible behind this.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Codes of slice w (32 elements) of a lane's share of a key row, as the halves
// of a matrix operand.  4 bits: half (v, h) of the operand holds element v + 4 h
// of the lane's 8, times 16 for odd v.  8 bits: elements 0 2 | 1 3 | 4 6 | 5 7.
template <int BITS>
__device__ __forceinline__ f16x8 key_operand(const uint32_t* k, int w) {
  if constexpr (BITS == 4) {
    const uint32_t a = k[w], b = a >> 8;
    return operand(a & 0x000f000fu, a & 0x00f000f0u, b & 0x000f000fu, b & 0x00f000f0u);
  } else {
    const uint32_t a = k[2 * w], b = k[2 * w + 1];
    return operand(a & 0x00ff00ffu, __builtin_amdgcn_perm(0u, a, 0x0c030c01u), b & 0x00ff00ffu,
                   __builtin_amdgcn_perm(0u, b, 0x0c030c01u));
  }
}

// Byte `byte` of the shares of two tokens, side by side in half words.
template <int WORDS>
__device__ __forceinline__ uint32_t byte_pair(const uint32_t (&a)[WORDS], const uint32_t (&b)[WORDS], int byte) {
  const uint32_t sel = 0x0c000c00u | (uint32_t)(byte % 4) | (uint32_t)(4 + byte % 4) << 16;
  return __builtin_amdgcn_perm(b[byte / 4], a[byte / 4], sel);
}

// (c - half) 2^-9 of two codes that lie in the low bits (SHIFT = 0) or one
// nibble higher (SHIFT = 4) of half words: exact, and normal numbers, which
// the matrix instruction adds up without loss.
template <int BITS, int SHIFT>
__device__ __forceinline__ uint32_t centred(uint32_t codes) {
  const _Float16 up = (_Float16)(SHIFT ? 0x1p11f : 0x1p15f);
  const _Float16 mid = (_Float16)(BITS == 4 ? -8.0f / 512 : -128.0f / 512);
  const f16x2 v = __builtin_elementwise_fma(__builtin_bit_cast(f16x2, codes), f16x2{up, up}, f16x2{mid, mid});
  return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ void store_out4(const KvRows& out, int64_t e, f32x4 v) {
  u32x2 w;
  if (out.dtype == kKvF16) {
    w.x = f32_to_f16(v.x) | f32_to_f16(v.y) << 16;
    w.y = f32_to_f16(v.z) | f32_to_f16(v.w) << 16;
  } else {
    w.x = f32_to_bf16(v.x) | f32_to_bf16(v.y) << 16;
    w.y = f32_to_bf16(v.z) | f32_to_bf16(v.w) << 16;
  }
  *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(out.p) + e) = w;
}

// The operand of value tile i (elements 16 i + 0..15) from a lane's shares of 8 tokens.
template <int BITS, int WORDS>
__device__ __forceinline__ f16x8 value_operand(const uint32_t (&v)[2][4][WORDS], int i) {
  const int byte = i * BITS / 8;
  auto half = [&](int s, int r) {
    const uint32_t c = byte_pair(v[s][r], v[s][r + 1], byte);
    if constexpr (BITS == 8) return centred<8, 0>(c);
    else return i & 1 ? centred<4, 4>(c & 0x00f000f0u) : centred<4, 0>(c & 0x000f000fu);
  };
  return operand(half(0, 0), half(0, 2), half(1, 0), half(1, 2));
}

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}
// op over aligned runs of LANES = 4 .. 32 lanes, the result in every lane of the run.
template <int LANES, typename Op>
__device__ __forceinline__ float run_reduce(float v, Op op) {
  v = op(v, dpp<0xB1>(v));                            // quad_perm [1,0,3,2]
  v = op(v, dpp<0x4E>(v));                            // quad_perm [2,3,0,1]
  if constexpr (LANES >= 8) v = op(v, dpp<0x141>(v));   // lane i <-> 7-i within 8
  if constexpr (LANES >= 16) v = op(v, dpp<0x140>(v));  // lane i <-> 15-i within 16
  if constexpr (LANES >= 32)
    v = op(v, __builtin_bit_cast(float, __builtin_amdgcn_ds_swizzle(__builtin_bit_cast(int, v), 0x401F)));
  return v;
}

// op over a wave, the same in all lanes.
template <typename Op>
__device__ __forceinline__ float wave_reduce(float v, Op op) {
  v = run_reduce<32>(v, op);
  auto lane = [v](int i) {
    return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), i));
  };
  return op(lane(0), lane(32));
}

// Query rows of a block in LDS, as matrix operands.
template <int BITS, int D, int G, int ROWS>
struct QueryRows {
  static constexpr int kSlices = D / 32, kGroups = D / G, kRuns = D / 8;
  f16x8 op[ROWS / 16][kSlices][64];
  float qs[ROWS][kGroups];   // sums of a row's elements over a group, * 2^-24

  // Elements `run` of row row0 + r of a (sequence, K/V head) with `rows` rows; 0 behind the last.
  __device__ __forceinline__ u32x4 load(const KvAttnArgs& a, const Seq& sq, int hk, int row, int rows, int run) const {
    if (row >= rows) return u32x4{0, 0, 0, 0};
    const int i = row / a.heads_per_kv, h = row - i * a.heads_per_kv;
    return *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(a.q.p) + (int64_t)(sq.first + i) * a.q.row_stride +
                                           (int64_t)(hk * a.heads_per_kv + h) * a.q.head_stride + run * 8);
  }
  static __device__ __forceinline__ void widen(u32x4 raw, int dtype, float* x) {
    if (dtype == kKvF16) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = f16_to_f32(j & 1 ? raw[j / 2] >> 16 : raw[j / 2] & 0xffffu);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(j & 1 ? raw[j / 2] & 0xffff0000u : raw[j / 2] << 16);
    }
  }
  // Elements x of a row, times 2^up, to their places.
  __device__ __forceinline__ void put(const float* x, int up, int r, int run) {
    _Float16 e[8];
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      e[j] = (_Float16)ldexpf(x[j], up);
      sum += (float)e[j];
    }
    sum = run_reduce<G / 8>(sum, [](float u, float v) { return u + v; });
    f16x8 o;
    if constexpr (BITS == 4) {
      const _Float16 low = (_Float16)0.0625f;   // codes one nibble higher count 16 times
      o = f16x8{e[0], e[4], e[1] * low, e[5] * low, e[2], e[6], e[3] * low, e[7] * low};
    } else {
      o = f16x8{e[0], e[2], e[1], e[3], e[4], e[6], e[5], e[7]};
    }
    op[r / 16][run / 4][run % 4 * 16 + r % 16] = o;
    // an infinite or NaN element makes every score of its row NaN here (infinity
    // less infinity in the softmax), also where all would be minus infinity
    if (run % (G / 8) == 0) qs[r][run / (G / 8)] = sum * 0x1p-24f + (sum - sum);
  }

  // All rows, each times a power of two; a row's size is its largest finite
  // element.  Where no row is 2^10 times smaller than the largest, whose size comes
  // into [2^14, 2^15), all have that one's power and one factor from raw scores to
  // log2 units, which is returned.  Else (`uneven`) every row has its own power,
  // which brings its own size there, and that factor times factor[row].  Either
  // way an element is off by 2^-25 of its row's size at most (4-bit codes: an odd
  // one enters as a sixteenth, and halves end at 2^-24).
  // A row's whole factor is kept to 2^100, so that products with a step are finite:
  // beyond (size times scale past 2^91) two scores are equal or differ by 2^30 and
  // more, cut or not (elements go down to 2^-25 of the size, keys to 2^-24), and one
  // key has all the weight.  Below 2^-80 it is kept too: scores under 2^-50 weigh
  // the same.
  // tops: two floats per wave.
  template <int THREADS>
  __device__ __forceinline__ float stage(const KvAttnArgs& a, const Seq& sq, int hk, int row0, int rows, float* tops,
                                         float (&factor)[ROWS], bool& uneven) {
    constexpr int kUnits = ROWS * kRuns, kPasses = (kUnits + THREADS - 1) / THREADS, kWaves = THREADS / 64;
    constexpr int kMost = 100, kLeast = -80, kMiddle = (kMost + kLeast) / 2;
    static_assert(kUnits % 64 == 0, "whole waves");
    u32x4 raw[kPasses];
#pragma unroll
    for (int pass = 0; pass < kPasses; ++pass) {
      const int unit = pass * THREADS + threadIdx.x;
      raw[pass] = unit < kUnits ? load(a, sq, hk, row0 + unit / kRuns, rows, unit % kRuns) : u32x4{0, 0, 0, 0};
    }
    auto larger = [](float u, float v) { return fmaxf(u, v); };
    auto smaller = [](float u, float v) { return fminf(u, v); };
    auto largest = [&](int pass) {   // finite element of this lane's 8
      float x[8], m = 0.0f;
      widen(raw[pass], a.q.dtype, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) m = fabsf(x[j]) < INFINITY ? fmaxf(m, fabsf(x[j])) : m;
      return m;
    };
    float top = 0.0f, least = INFINITY;   // of all runs of 8 elements; least: of those that are not all 0
#pragma unroll
    for (int pass = 0; pass < kPasses; ++pass) {
      const float m = largest(pass);
      top = fmaxf(top, m);
      least = m > 0.0f ? fminf(least, m) : least;
    }
    tops[threadIdx.x / 64] = wave_reduce(top, larger);
    tops[kWaves + threadIdx.x / 64] = wave_reduce(least, smaller);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
      top = fmaxf(top, tops[i]);
      least = fminf(least, tops[kWaves + i]);
    }
    auto uniform = [](float v) { return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(v))); };
    top = uniform(top);
    // a row is as large as its largest run: this is more than it takes, and yet never so for queries of one spread
    uneven = uniform(least) < top * 0x1p-10f;
    const int up = 15 - __builtin_amdgcn_frexp_expf(top);
    if (uneven) {
#pragma unroll
      for (int pass = 0; pass < kPasses; ++pass) {
        const int unit = pass * THREADS + threadIdx.x;
        const float size = run_reduce<kRuns>(largest(pass), larger);
        if (unit >= kUnits) break;
        const int exponent = a.scale_exp + 24 - (size > 0.0f ? 15 - __builtin_amdgcn_frexp_expf(size) : up);
        const int kept = min(max(exponent, kLeast), kMost);
        float x[8];
        widen(raw[pass], a.q.dtype, x);
        // a row under kLeast comes in smaller; one past kMost stays in f16's range
        put(x, a.scale_exp + 24 - max(exponent, kLeast), unit / kRuns, unit % kRuns);
        if (unit % kRuns == 0) factor[unit / kRuns] = ldexpf(1.0f, kept - kMiddle);
      }
      return ldexpf(a.scale_log2, kMiddle);
    }
#pragma unroll
    for (int pass = 0; pass < kPasses; ++pass) {
      const int unit = pass * THREADS + threadIdx.x;
      float x[8];
      if (unit >= kUnits) break;
      widen(raw[pass], a.q.dtype, x);
      put(x, up, unit / kRuns, unit % kRuns);
    }
    return ldexpf(a.scale_log2, min(a.scale_exp + 24 - up, kMost));
  }
};

// What the softmax of a tile of 32 keys takes of its parameters, in LDS.
template <int D, int G>
struct TileParams {
  static constexpr int kGroups = D / G;
  f16x8 sums[64];                       // operand of the sums that need no code: rows of zeros, of steps, of ones
  float step[2][2][16][kGroups];        // key step * row factor; value step * einv
  float kzero[2][16][kGroups];

  // Eight groups leave no row of 16 for the ones.
  static constexpr bool kSumRow = 2 * kGroups < 16;
  // Lane `i` of what put() does not write: the row of ones, and zeros behind it.
  __device__ __forceinline__ void clear(int i) {
    const uint32_t one = kSumRow && i % 16 == 2 * kGroups ? 0x3c003c00u : 0u;
    sums[i] = operand(one, one, one, one);
  }
};

// A tile's parameter words in one wave's registers: word 64 i + lane of [keys,
// values][half][token][group].
template <int D, int G>
struct ParamWords {
  static constexpr int kGroups = D / G;
  uint32_t word[kGroups];

  __device__ __forceinline__ void load(const KvCache& c, int64_t row0, int64_t row1) {
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      const uint32_t w = i * 64 + threadIdx.x % 64, run = w / (16 * kGroups);
      const uint32_t* from = run & 2 ? c.v_params : c.k_params;
      word[i] = from[(run & 1 ? row1 : row0) * kGroups + w % (16 * kGroups)];
    }
  }
  // Words of keys that no row of the block sees become 0: nobody need have
  // written their slots, and what lies there would reach the products (0 * NaN)
  // and the normaliser of the steps.  The rows see the keys from `lo` to `end`
  // and the first `sinks`.
  __device__ __forceinline__ void clear_unseen(int tb, int end, int lo, int sinks, uint32_t ok) {
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      const int w = i * 64 + threadIdx.x % 64, s = w / (16 * kGroups) & 1, j = tb + 16 * s + w % (16 * kGroups) / kGroups;
      if (!(j < end && (j >= lo || j < sinks) && (ok >> s & 1u))) word[i] = 0u;
    }
  }
  __device__ __forceinline__ float largest_step() const {   // of this lane's values
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < kGroups; ++i)
      if (i * 64 + threadIdx.x % 64 >= 32 * kGroups) top = fmaxf(top, f16_to_f32(word[i] & 0xffffu));
    return top;
  }
  __device__ __forceinline__ void put(TileParams<D, G>& to, float rf, float einv) const {
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      const int w = i * 64 + threadIdx.x % 64, at = w % (32 * kGroups);   // [half][token][group]
      const bool value = w >= 32 * kGroups;
      (&to.step[0][0][0][0])[w] = f16_to_f32(word[i] & 0xffffu) * (value ? einv : rf);
      if (value) {
        const int g = at % kGroups, token = at / kGroups, j = token / 16 * 4 + token % 4;
        uint16_t* zeros = reinterpret_cast<uint16_t*>(&to.sums[token % 16 / 4 * 16 + g]);
        uint16_t* steps = reinterpret_cast<uint16_t*>(&to.sums[token % 16 / 4 * 16 + kGroups + g]);
        zeros[j] = (uint16_t)(word[i] >> 16);
        steps[j] = (uint16_t)word[i];
      } else {
        (&to.kzero[0][0][0])[at] = f16_to_f32(word[i] >> 16);
      }
    }
  }
};

// The power of two that value steps are multiplied with, so that products of a
// probability and a step stay in f16's range: the largest step seen comes into
// [1/2, 1).  It changes when a larger one comes.
struct StepScale {
  float einv = 1.0f, limit = 0.0f;
  // step: one of the coming values' steps per lane, all of them over the wave.
  // True: einv has changed.
  __device__ __forceinline__ bool see(float step) {
    if (!__any(step > limit)) return false;
#pragma unroll
    for (int i = 1; i < 64; i *= 2) step = fmaxf(step, __shfl_xor(step, i));
    const int e = (int)(__float_as_uint(step) >> 23) - 127 + 1;
    einv = ldexpf(1.0f, -e);
    limit = ldexpf(1.0f, e);
    return true;
  }
};

// What the many-row step reads from LDS ahead of its use: left to itself the
// compiler puts each read right before its two matrix instructions, and the
// wave waits for it (2048 rows after 16384 keys of 128 elements: 743 us, with
// operands ahead 674, parameters too 665; where that spills it costs more: 64
// elements 334 us without parameters, 430 with).  kOperands: matrix operands;
// kAll: a half's parameters too.
enum class Ahead { kNothing, kOperands, kAll };
constexpr Ahead ahead(int D, int G) {
  return D == 128 && G == 128 ? Ahead::kAll : D / G <= (D == 64 ? 1 : 2) ? Ahead::kOperands : Ahead::kNothing;
}

// The state of a wave: 16 NT query rows against the keys seen so far.
template <int BITS, int D, int G, int NT>
struct Wave {
  using Params = TileParams<D, G>;
  static constexpr int kSlices = D / 32, kTiles = D / 16, kGroups = D / G;
  static constexpr float kHalf = BITS == 4 ? 8.0f : 128.0f;
  f16x8 q[NT][kSlices];          // query rows as matrix operands
  float qs[NT][kGroups];         // sum of a row's q over a group, in log2 units of score (over the row's factor)
  int lo[NT], hi[NT];            // visible keys: j <= hi and (j >= lo or j < sinks)
  f32x4 o[NT][kTiles];           // sum of p step einv (c - kHalf) 2^-9
  f32x4 st[NT];                  // rows: g: sum p zero; kGroups + g: sum p step; 2 kGroups: sum p
  float l[NT];                   // (!kSumRow) this lane's part of sum p
  float mb[NT];                  // running maximum (log2) - kPeak
  bool none[NT];                 // no key seen yet
  bool fresh;                    // `none` of some row of the wave
  // Rows have factors of their own (QueryRows::stage): scores then come without
  // the running maximum, times 1 / factor, and are put right where masks are set,
  // in a branch that steps of ordinary queries inside every row's view pass by
  // (2048 rows after 16384 keys, and ragged prompts at 64 elements: 667 and 335 us;
  // with one power of two for a block, which took bits from its smaller rows, 661
  // and 331; with the maximum in each row's own units 664 and 346; with a walk over
  // the keys for every range of sizes 697 and 368).
  bool uneven;
  const float* factor;           // of the wave's rows, in LDS
  float einv;                    // of o

  // Rows row0 + first .. of the block's staged rows; rf: from raw scores to log2
  // units, but for the rows' own factors where they have some.
  template <int ROWS>
  __device__ __forceinline__ void begin(const KvAttnArgs& a, const Seq& sq, const QueryRows<BITS, D, G, ROWS>& from,
                                        float rf, bool own_factors, const float* factors, int row0, int first, int rows) {
    const int n = threadIdx.x % 16, lane = threadIdx.x % 64;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int r = first + t * 16 + n, row = row0 + r;
      const bool exists = row < rows;
      const int pos = (int)((uint32_t)sq.pos + (uint32_t)(row / a.heads_per_kv));   // may wrap where the row does not exist
      hi[t] = !a.causal || !exists ? sq.len - 1 : pos < sq.len ? pos : sq.len - 1;
      lo[t] = exists ? window_start(a.window, pos) : 0;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) qs[t][g] = from.qs[r][g] * rf;
#pragma unroll
      for (int w = 0; w < kSlices; ++w) q[t][w] = from.op[first / 16 + t][w][lane];
      st[t] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < kTiles; ++i) o[t][i] = f32x4{0, 0, 0, 0};
      mb[t] = 0.0f;
      l[t] = 0.0f;
      none[t] = true;
    }
    fresh = true;
    uneven = own_factors;
    factor = factors + first;
    einv = 1.0f;
  }

  // o in units of another power of two.
  __device__ __forceinline__ void set_scale(float e) {
    if (e == einv) return;
    const float ratio = e / einv;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < kTiles; ++i) o[t][i] *= ratio;
    einv = e;
  }

  // SUB tiles of 32 keys, at tokens tb.  key(u, s, w): operand of slice w of half
  // s of tile u; value(u, i): operand of value tile i; params(u): the tile's
  // parameters; whole: every row sees all of the keys, and rows have no
  // factors of their own; ok: bit s: half s lies in a page of the cache.
  template <int SUB, typename Key, typename Value, typename P>
  __device__ __forceinline__ void step(Key&& key, Value&& value, P&& params, const int (&tb)[SUB], bool whole, int len,
                                       const uint32_t (&ok)[SUB], int sinks) {
    const int lane = threadIdx.x % 64, quad = lane / 16;
    // scores in log2 units less the running maximum; half h % 2 of tile h / 2
    float y[SUB][NT][2][4];
    float less[NT];   // what scores come without
#pragma unroll
    for (int i = 0; i < NT; ++i) less[i] = uneven ? 0.0f : mb[i];
    constexpr int kHalves = 2 * SUB;
    constexpr Ahead kAhead = SUB > 1 ? ahead(D, G) : Ahead::kNothing;
    f16x8 ops[2][kSlices];
    f32x4 acc[2][kGroups][NT];
    float ks[2][kGroups][4], kz[2][kGroups][4];
    auto keys = [&](int h) {
#pragma unroll
      for (int w = 0; w < kSlices; ++w) ops[h % 2][w] = key(h / 2, h % 2, w);
    };
    auto factors = [&](int h, int g) {
      const Params& x = params(h / 2);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        ks[h % 2][g][j] = x.step[0][h % 2][quad * 4 + j][g];
        kz[h % 2][g][j] = x.kzero[h % 2][quad * 4 + j][g];
      }
    };
    auto scores = [&](int h, int g) {
      if constexpr (kAhead != Ahead::kAll) factors(h, g);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const float z = fmaf(kz[h % 2][g][j], qs[i][g], g == 0 ? -less[i] : y[h / 2][i][h % 2][j]);
          y[h / 2][i][h % 2][j] = fmaf(ks[h % 2][g][j], acc[h % 2][g][i][j], z);
        }
    };
    if constexpr (kAhead != Ahead::kNothing) keys(0);
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
      if constexpr (kAhead != Ahead::kNothing) {
        if constexpr (kAhead == Ahead::kAll)
#pragma unroll
          for (int g = 0; g < kGroups; ++g) factors(h, g);
        if (h + 1 < kHalves) keys(h + 1);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
#pragma unroll
        for (int i = 0; i < NT; ++i) acc[h % 2][g][i] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int w = g * G / 32; w < (g + 1) * G / 32; ++w) {
          const f16x8 op = kAhead != Ahead::kNothing ? ops[h % 2][w] : key(h / 2, h % 2, w);
#pragma unroll
          for (int i = 0; i < NT; ++i) acc[h % 2][g][i] = mfma(op, q[i][w], acc[h % 2][g][i]);
        }
        if constexpr (kAhead == Ahead::kNothing) scores(h, g);
        else if (h > 0) scores(h - 1, g);
      }
    }
    if constexpr (kAhead != Ahead::kNothing)
#pragma unroll
      for (int g = 0; g < kGroups; ++g) scores(kHalves - 1, g);
    if (!whole) {
      if (uneven) {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const float f = factor[i * 16 + lane % 16];
#pragma unroll
          for (int u = 0; u < SUB; ++u)
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
              for (int j = 0; j < 4; ++j) y[u][i][s][j] = fmaf(y[u][i][s][j], f, -mb[i]);
        }
      }
#pragma unroll
      for (int u = 0; u < SUB; ++u)
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int at = tb[u] + 16 * s + quad * 4 + j;
            const bool there = at < len && (ok[u] >> s & 1u);
#pragma unroll
            for (int i = 0; i < NT; ++i)
              if (!(there && at <= hi[i] && (at >= lo[i] || at < sinks))) y[u][i][s][j] = -INFINITY;
          }
    }
    float top[NT];
    bool above = fresh;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      top[i] = -INFINITY;
#pragma unroll
      for (int u = 0; u < SUB; ++u)
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int j = 0; j < 4; ++j) top[i] = fmaxf(top[i], y[u][i][s][j]);
      above |= top[i] > kPeak + kSlack;
    }
    if (__any(above)) {
      fresh = false;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        float m = top[i];
        m = fmaxf(m, __shfl_xor(m, 16));
        m = fmaxf(m, __shfl_xor(m, 32));
        const bool any = m > -INFINITY;
        // a row's first keys set its maximum, later ones only raise it
        float up = !any ? 0.0f : none[i] ? m - kPeak : fmaxf(m - kPeak, 0.0f);
        // where floats of m's size lie 16 apart, m - kPeak is m - 16, and 2^16 no half
        up = m - up > kPeak + kSlack ? m : up;
        const float alpha = none[i] ? 1.0f : __builtin_amdgcn_exp2f(-up);   // nothing to scale yet
        mb[i] += up;
        none[i] = none[i] && !any;
        fresh |= none[i];
        st[i] *= alpha;
        l[i] *= alpha;
#pragma unroll
        for (int j = 0; j < kTiles; ++j) o[i][j] *= alpha;
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
          for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int j = 0; j < 4; ++j) y[u][i][s][j] -= up;
      }
      fresh = __any(fresh);
    }
    constexpr int kDeep = D == 64 ? 2 : 4;
    f16x8 vops[kDeep];
    if constexpr (kAhead != Ahead::kNothing) {
#pragma unroll
      for (int d = 0; d < kDeep; ++d) vops[d] = value(0, d);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int u = 0; u < SUB; ++u) {
      const Params& x = params(u);
      const f16x8 sums = x.sums[lane];
      f16x8 pv[NT][kGroups];
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        f16x8 p;
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float e = __builtin_amdgcn_exp2f(y[u][i][s][j]);
            p[4 * s + j] = (_Float16)e;
            if constexpr (!Params::kSumRow) l[i] += e;
#pragma unroll
            for (int g = 0; g < kGroups; ++g) pv[i][g][4 * s + j] = (_Float16)(e * x.step[1][s][quad * 4 + j][g]);
          }
        st[i] = mfma(sums, p, st[i]);
      }
      if constexpr (kAhead == Ahead::kNothing) {
#pragma unroll
        for (int d = 0; d < kTiles; ++d) {
          const f16x8 op = value(u, d);
#pragma unroll
          for (int i = 0; i < NT; ++i) o[i][d] = mfma(op, pv[i][d * 16 / G], o[i][d]);
        }
      } else {
#pragma unroll
        for (int d = 0; d < kTiles; ++d) {
          const f16x8 op = vops[d % kDeep];
          if (d + kDeep < kTiles) vops[d % kDeep] = value(u, d + kDeep);
          else if (u + 1 < SUB) vops[d % kDeep] = value(u + 1, d + kDeep - kTiles);
          __builtin_amdgcn_sched_barrier(0x406);
#pragma unroll
          for (int i = 0; i < NT; ++i) o[i][d] = mfma(op, pv[i][d * 16 / G], o[i][d]);
        }
      }
    }
  }

  // Row `row` of the sums' result for this lane's query row, from the lane that holds it.
  __device__ __forceinline__ float sum_of(int t, int row) const {
    return __shfl(st[t][row % 4], (int)(threadIdx.x % 16) + 16 * (row / 4));
  }

  // The running maximum of tile t's rows as the join takes it.
  __device__ __forceinline__ float maximum(int t) const { return none[t] ? kLowest : mb[t]; }

  // The sum of probabilities of tile t's rows; the outputs in the same units, in place of o.
  __device__ __forceinline__ float finish(int t) {
    const float up = 0x1p9f / einv;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const float z = fmaf(kHalf, sum_of(t, kGroups + g), sum_of(t, g));
#pragma unroll
      for (int i = g * G / 16; i < (g + 1) * G / 16; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) o[t][i][r] = fmaf(o[t][i][r], up, z);
    }
    if constexpr (Params::kSumRow) return sum_of(t, 2 * kGroups);
    float sum = l[t] + __shfl_xor(l[t], 16);
    return sum + __shfl_xor(sum, 32);
  }
};

// What a block works on, and the bounds over a range of its rows: a tile inside
// all of them needs no mask, one outside all of them nothing.
struct Block {
  Seq sq;
  Span span;
  int b, hk, rb, split, row0, rows, active, t0, t1;
  const int32_t* table;
};
struct Bounds {
  int hi_min, hi_max, lo_min, lo_max;
};

// grid.x: K/V head fastest, then sequence, block of rows (the last rows first:
// under a causal mask they have the most keys), split: long blocks start early.
// False: the block has nothing to do.
__device__ __forceinline__ bool block_of(const KvAttnArgs& a, int block_rows, Block& k) {
  uint32_t id = blockIdx.x;
  k.hk = (int)(id % (uint32_t)a.c.kv_heads);
  id /= (uint32_t)a.c.kv_heads;
  k.b = (int)(id % (uint32_t)a.b.seqs);
  id /= (uint32_t)a.b.seqs;
  k.rb = a.plan.row_blocks - 1 - (int)(id % (uint32_t)a.plan.row_blocks);
  k.split = (int)(id / (uint32_t)a.plan.row_blocks);
  k.sq = sequence(a, k.b);
  k.rows = k.sq.computed * a.heads_per_kv;
  k.row0 = k.rb * block_rows;
  if (k.row0 >= k.rows) return false;
  const int last = min(k.row0 + block_rows, k.rows) - 1;
  k.span = key_span(a, k.sq.len, (int64_t)k.sq.len - k.sq.pos, k.row0 / a.heads_per_kv, last / a.heads_per_kv);
  k.active = (k.span.tiles + a.plan.split_tiles - 1) / a.plan.split_tiles;
  k.t0 = k.split * a.plan.split_tiles;
  k.t1 = min(k.t0 + a.plan.split_tiles, k.span.tiles);
  k.table = a.b.page_table + (int64_t)k.b * a.b.table_stride;
  return k.split == 0 || k.split < k.active;
}
__device__ __forceinline__ Bounds bounds_of(const KvAttnArgs& a, const Block& k, int first, int last) {
  const int p0 = k.sq.pos + first / a.heads_per_kv, p1 = k.sq.pos + last / a.heads_per_kv;
  return Bounds{a.causal ? p0 : k.sq.len - 1, a.causal ? p1 : k.sq.len - 1, window_start(a.window, p0),
                window_start(a.window, p1)};
}
__device__ __forceinline__ bool tile_seen(const Bounds& r, int tb, int sinks) {
  return tb <= r.hi_max && (tb + kTile > r.lo_min || tb < sinks);
}
__device__ __forceinline__ bool tile_whole(const Bounds& r, int tb, int len, uint32_t ok, int sinks) {
  return tb + kTile - 1 <= r.hi_min && tb + kTile <= len && ok == 3u && (tb >= r.lo_max || tb + kTile <= sinks);
}

__device__ __forceinline__ void store_out8(const KvRows& out, int64_t e, const float* v) {
  u32x4 w;
  if (out.dtype == kKvF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = f32_to_f16(v[2 * i]) | f32_to_f16(v[2 * i + 1]) << 16;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = f32_to_bf16(v[2 * i]) | f32_to_bf16(v[2 * i + 1]) << 16;
  }
  *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(out.p) + e) = w;
}

// The splits' results pass between blocks on different dies, whose L2 caches are
// not coherent: they are stored and loaded as agent-scope atomics, which go
// through to the common memory.  (Fences of that scope write back and drop the
// whole L2 instead: with one per block a decode step of 64 sequences took 150
// us in place of 46.)  Their order against the arrival counter is gfx950's, not
// the language's, which orders no relaxed atomics: an agent-scope store (sc1) has
// left the die's L2 when vmcnt counts it down, so behind s_waitcnt vmcnt(0) of
// every wave, and the barrier, the counter is only reached by results that are
// there for all dies; and an agent-scope load (sc1) takes no older line from its
// own L2.
__device__ __forceinline__ void put_shared(float* p, float v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float get_shared(const float* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Behind the stores of a split's results: the last of the splits of a block's
// rows to arrive joins them all, in the order of the splits.  It leaves the
// counter 0 for the next call.  `word`: LDS.
template <int D, int THREADS, int kBatch>
__device__ __forceinline__ void join_splits(const KvAttnArgs& a, const Block& k, int block_rows, uint32_t* word) {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // this wave's results have arrived
  __syncthreads();                                    // and the other waves'
  if (threadIdx.x == 0) {
    uint32_t* counter = a.counters + ((int64_t)k.b * a.c.kv_heads + k.hk) * a.plan.row_blocks + k.rb;
    *word = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (*word == (uint32_t)k.active - 1) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  if (*word != (uint32_t)k.active - 1) return;
  constexpr int kRuns = D / 8;
  const int rows = min(block_rows, k.rows - k.row0);
  for (int unit = threadIdx.x; unit < rows * kRuns; unit += THREADS) {
    const int row = k.row0 + unit / kRuns, run = unit % kRuns;
    const int64_t at = part_index(a, k.b, k.hk, a.plan.row_blocks * block_rows, row, 0);
    const float* ml = a.part_ml + at * 2;
    const float* po = a.part_o + at * D + run * 8;
    float top = kLowest, sum = 0.0f, v[8] = {};
    // kBatch splits' loads in flight together; behind the last split that one again, with weight 0
    for (int s0 = 0; s0 < k.active; s0 += kBatch) {
      float m[kBatch], l[kBatch], o[kBatch][8], t = top;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int s = min(s0 + i, k.active - 1);
        m[i] = get_shared(ml + 2 * s);
        l[i] = get_shared(ml + 2 * s + 1);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[i][e] = get_shared(po + (int64_t)s * D + e);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) t = fmaxf(t, m[i]);
      const float down = __builtin_amdgcn_exp2f(top - t);
      top = t;
      sum *= down;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= down;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const float f = s0 + i < k.active ? __builtin_amdgcn_exp2f(m[i] - top) : 0.0f;
        sum = fmaf(l[i], f, sum);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = fmaf(o[i][e], f, v[e]);
      }
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    const int i = row / a.heads_per_kv, h = k.hk * a.heads_per_kv + row - i * a.heads_per_kv;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= inv;
    store_out8(a.out, (int64_t)(k.sq.first + i) * a.out.row_stride + (int64_t)h * a.out.head_stride + run * 8, v);
  }
}

// ------------------------------------------------------------------ few rows
// The NW waves of a block share its 16 NT rows and take turns over the keys:
// wave w has the tiles w, w + NW, ...  Loads go to registers, the next tile's
// in flight during the current one's arithmetic; no barrier in the loop.  At
// the end the waves' results meet in LDS.
template <int BITS, int D, int G, int NT, int NW>
struct FewLds {
  static constexpr int kRows = NT * 16, kStride = D + 4;
  QueryRows<BITS, D, G, kRows> q;
  float top[2 * NW];
  float factor[kRows];
  float m[NW][kRows], l[NW][kRows];
  union {
    TileParams<D, G> params;    // in the wave's loop
    float o[kRows][kStride];    // behind it
  } wave[NW];
};

// Waves per SIMD that the registers leave room for.  With 8 waves a block there
// are two at least, and then groups of 32 spill: 1 register at 4 bits, 128
// elements and two tiles, 45 at 4 bits and 256 elements, 46 at 8 bits, 128
// elements and two tiles.  64 sequences of 4096 keys, groups of 32 / 128: 83 / 62,
// 162 / 103 (one row of 4 heads) and 147 / 104 us; without spills, at 4 bits, 128
// elements and one tile, 66 / 56.
constexpr int few_min_waves(int BITS, int D, int G, int NT) {
  if (NT == 1) return D == 64 ? (BITS * (64 / G) > 8 ? 3 : 4) : D == 128 ? (BITS == 4 && G > 32 ? 3 : 2) : BITS == 4 && G > 32 ? 2 : 1;
  return BITS * (128 / G) < 32 ? 2 : 1;
}

template <int BITS, int D, int G, int NT, int NW>
__global__ __launch_bounds__(NW * 64, few_min_waves(BITS, D, G, NT)) void k_kv_attention_few(KvAttnArgs a) {
  using W = Wave<BITS, D, G, NT>;
  using Lds = FewLds<BITS, D, G, NT, NW>;
  extern __shared__ __align__(16) uint8_t shared[];
  Lds& lds = *reinterpret_cast<Lds*>(shared);
  Block k;
  if (!block_of(a, Lds::kRows, k)) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  int t = k.t0 + wave;
  Tile<BITS, D, G> x, y;
  ParamWords<D, G> x_words, y_words;
  uint32_t x_ok = 0, y_ok = 0;
  // past the last tile the loads repeat it; nothing uses the copy
  auto token = [&](int at) { return k.span.token(min(at, k.t1 - 1)); };
  Pages pages = {{-1, -1}};   // of the next tile to load
  auto fetch = [&](Tile<BITS, D, G>& into, ParamWords<D, G>& words, uint32_t& ok, int at) {
    const Halves h = tile_halves(a.c, pages, k.hk, token(at));
    ok = pages.ok();
    load_tile(into, a.c, h);
    words.load(a.c, h.row[0], h.row[1]);
    pages = tile_pages(a.c, k.table, k.sq.len, token(at + NW));
  };
  if (t < k.t1) {
    pages = tile_pages(a.c, k.table, k.sq.len, token(t));
    fetch(x, x_words, x_ok, t);
  }
  TileParams<D, G>& params = lds.wave[wave].params;
  params.clear(threadIdx.x % 64);
  bool uneven;
  const float rf = lds.q.template stage<NW * 64>(a, k.sq, k.hk, k.row0, k.rows, lds.top, lds.factor, uneven);
  __syncthreads();
  W w;
  w.begin(a, k.sq, lds.q, rf, uneven, lds.factor, k.row0, 0, k.rows);
  StepScale scale;
  const Bounds r = bounds_of(a, k, k.row0, min(k.row0 + Lds::kRows, k.rows) - 1);
  auto work = [&](const Tile<BITS, D, G>& from, ParamWords<D, G>& words, uint32_t page_ok) {
    const int tb[1] = {k.span.token(t)};
    if (tile_seen(r, tb[0], a.sinks)) {
      const uint32_t ok[1] = {page_ok};
      const bool whole = !uneven && tile_whole(r, tb[0], k.sq.len, page_ok, a.sinks);
      if (!whole) words.clear_unseen(tb[0], k.span.end, r.lo_min, a.sinks, page_ok);
      if (scale.see(words.largest_step())) w.set_scale(scale.einv);
      wave_sync();
      words.put(params, rf, scale.einv);
      wave_sync();
      w.template step<1>([&](int, int s, int i) { return key_operand<BITS>(from.k[s], i); },
                         [&](int, int i) { return value_operand<BITS>(from.v, i); },
                         [&](int) -> const TileParams<D, G>& { return params; }, tb, whole, k.sq.len, ok, a.sinks);
    }
    t += NW;
  };
  while (t < k.t1) {   // two buffers taking turns: a copy would wait for the loads in flight
    fetch(y, y_words, y_ok, t + NW);
    work(x, x_words, x_ok);
    if (t >= k.t1) break;
    fetch(x, x_words, x_ok, t + NW);
    work(y, y_words, y_ok);
  }
  const int n = threadIdx.x % 16, quad = threadIdx.x / 16 % 4;
  wave_sync();
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const float l = w.finish(i);
    const int row = i * 16 + n;
    if (quad == 0) {
      lds.m[wave][row] = w.maximum(i);
      lds.l[wave][row] = l;
    }
#pragma unroll
    for (int e = 0; e < W::kTiles; ++e) *reinterpret_cast<f32x4*>(&lds.wave[wave].o[row][e * 16 + quad * 4]) = w.o[i][e];
  }
  __syncthreads();
  constexpr int kRuns = D / 8;
#pragma unroll
  for (int pass = 0; pass * NW * 64 < Lds::kRows * kRuns; ++pass) {
    const int unit = pass * NW * 64 + threadIdx.x, r0 = unit / kRuns, run = unit % kRuns;
    const int row = k.row0 + r0;
    if (unit >= Lds::kRows * kRuns || row >= k.rows) break;
    float top = kLowest, sum = 0.0f, v[8] = {};
#pragma unroll
    for (int i = 0; i < NW; ++i) top = fmaxf(top, lds.m[i][r0]);
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      const float f = __builtin_amdgcn_exp2f(lds.m[i][r0] - top);
      sum = fmaf(lds.l[i][r0], f, sum);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = fmaf(lds.wave[i].o[r0][run * 8 + e], f, v[e]);
    }
    if (k.active <= 1) {
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;   // a row that sees nothing becomes 0
      const int i = row / a.heads_per_kv, h = k.hk * a.heads_per_kv + row - i * a.heads_per_kv;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= inv;
      store_out8(a.out, (int64_t)(k.sq.first + i) * a.out.row_stride + (int64_t)h * a.out.head_stride + run * 8, v);
    } else {
      const int64_t at = part_index(a, k.b, k.hk, a.plan.row_blocks * Lds::kRows, row, k.split);
      if (run == 0) {
        put_shared(a.part_ml + at * 2, top);
        put_shared(a.part_ml + at * 2 + 1, sum);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) put_shared(a.part_o + at * D + run * 8 + e, v[e]);
    }
  }
  if (k.active > 1) join_splits<D, NW * 64, 4>(a, k, Lds::kRows, reinterpret_cast<uint32_t*>(lds.top));
}

// ------------------------------------------------------------------ many rows
// Each of the NW waves of a block has its own 16 NT rows and all walk the same
// keys, two tiles of 32 a step.  The waves unpack the codes once, each a quarter
// of one tile, into matrix operands in LDS (two buffers, one barrier a step),
// and one wave the parameters into what the softmax uses; doing either per wave
// would cost as much as the softmax.  The block's query rows share one power of
// two (where their sizes allow it), so that a score in log2 units less the running
// maximum takes two multiply-adds: a key's step and the row factor are one number.
template <int BITS, int D, int G>
struct ManyTile {
  f16x8 k[2][D / 32][64];
  f16x8 v[D / 16][64];
  TileParams<D, G> params;
};
constexpr int kSub = 2;
template <int BITS, int D, int G, int NT, int NW>
struct ManyLds {
  static constexpr int kRows = NW * NT * 16;
  struct Step {
    ManyTile<BITS, D, G> tile[kSub];
    float einv;                         // of the values' steps
    uint32_t ok[kSub];                  // bit s: half s lies in a page of the cache
  };
  float top[2 * NW];
  float factor[kRows];
  union {
    QueryRows<BITS, D, G, kRows> q;     // before the first step
    Step step[2];
  };
};

// A wave's quarter of a tile in registers: half s = quarter / 2, part = quarter
// % 2 of its slices and bytes.
template <int BITS, int D, int G>
struct Quarter {
  using T = Tile<BITS, D, G>;
  static constexpr int kKeyWords = T::kKeyWords / 2;          // half of a lane's share of a key row
  static constexpr int kBytes = T::kUnitBytes / 2;            // half of its share of a value row
  static constexpr int kWords = kBytes < 4 ? 1 : kBytes / 4;
  uint32_t k[kKeyWords], v[4][kWords];

  __device__ __forceinline__ void load(const KvCache& c, const int32_t* table, int len, int hk, int tb, int quarter) {
    const uint32_t n = threadIdx.x % 16, quad = threadIdx.x / 16 % 4;
    const int s = quarter / 2, part = quarter % 2;
    const int64_t mine = half_row(c, half_page(c, table, len, tb + 16 * s), hk, tb + 16 * s);
    const uint8_t* kc = c.k_codes + mine * T::kRowBytes + part * (kKeyWords * 4);
    const uint8_t* vc = c.v_codes + mine * T::kRowBytes + part * kBytes;
    load_words<kKeyWords>(kc + n * T::kRowBytes + quad * (T::kRowBytes / 4), k);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const uint8_t* u = vc + (quad * 4 + r) * T::kRowBytes + n * T::kUnitBytes;
      if constexpr (kBytes == 1) v[r][0] = *u;
      else if constexpr (kBytes == 2) v[r][0] = *reinterpret_cast<const uint16_t*>(u);
      else load_words<kWords>(u, v[r]);
    }
  }

  __device__ __forceinline__ void unpack(ManyTile<BITS, D, G>& to, int quarter) const {
    const int lane = threadIdx.x % 64, s = quarter / 2, part = quarter % 2;
    constexpr int kSlices = D / 32 / 2;
#pragma unroll
    for (int w = 0; w < kSlices; ++w) to.k[s][part * kSlices + w][lane] = key_operand<BITS>(k, w);
    constexpr int kTiles = D / 16 / 2;
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      const int byte = i * BITS / 8;
      u32x2 h;
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const uint32_t c = byte_pair(v[2 * p], v[2 * p + 1], byte);
        if constexpr (BITS == 8) h[p] = centred<8, 0>(c);
        else h[p] = i & 1 ? centred<4, 4>(c & 0x00f000f0u) : centred<4, 0>(c & 0x000f000fu);
      }
      reinterpret_cast<u32x2*>(&to.v[part * kTiles + i][lane])[s] = h;
    }
  }

};

template <int BITS, int D, int G, int NT, int NW>
__global__ __launch_bounds__(NW * 64, D == 64 ? 3 : 2) void k_kv_attention_many(KvAttnArgs a) {
  using Lds = ManyLds<BITS, D, G, NT, NW>;
  using W = Wave<BITS, D, G, NT>;
  constexpr int SUB = kSub;
  extern __shared__ __align__(16) uint8_t shared[];
  Lds& lds = *reinterpret_cast<Lds*>(shared);
  Block k;
  if (!block_of(a, Lds::kRows, k)) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int lane = threadIdx.x % 64, n = lane % 16, quad = lane / 16;
  const int first = wave * NT * 16;

  bool uneven;
  const float rf = lds.q.template stage<NW * 64>(a, k.sq, k.hk, k.row0, k.rows, lds.top, lds.factor, uneven);
  __syncthreads();
  W w;
  w.begin(a, k.sq, lds.q, rf, uneven, lds.factor, k.row0, first, k.rows);
  __syncthreads();             // the steps overwrite the staged rows
  for (int i = threadIdx.x; i < 2 * SUB * 64; i += NW * 64)
    lds.step[i / (SUB * 64)].tile[i / 64 % SUB].params.clear(i % 64);
  __syncthreads();
  // a wave without rows works along on those of the block's last row
  const Bounds r = bounds_of(a, k, min(k.row0 + first, k.rows - 1), min(k.row0 + first + NT * 16, k.rows) - 1);
  const bool idle = k.row0 + first >= k.rows;

  // Each wave fetches and unpacks its quarter of one tile (of 8 waves) or of both
  // (of 4), the first one all parameters.
  constexpr int kMine = SUB * 4 / NW;
  const int quarter = wave % 4;
  auto mine = [&](int i) { return NW == 8 ? wave / 4 : i; };
  Quarter<BITS, D, G> codes[kMine];
  ParamWords<D, G> words[SUB];
  uint32_t ok[SUB];
  StepScale scale;                               // first wave: of the coming step's values
  auto token = [&](int t) { return k.span.token(min(t, k.t1 - 1)); };   // past the last tile: that one again
  auto fetch = [&](int t) {
#pragma unroll
    for (int i = 0; i < kMine; ++i) codes[i].load(a.c, k.table, k.sq.len, k.hk, token(t + mine(i)), quarter);
    if (wave == 0) {
#pragma unroll
      for (int u = 0; u < SUB; ++u) {
        const Pages pages = tile_pages(a.c, k.table, k.sq.len, token(t + u));
        const Halves h = tile_halves(a.c, pages, k.hk, token(t + u));
        words[u].load(a.c, h.row[0], h.row[1]);
        ok[u] = pages.ok();
      }
    }
  };
  auto unpack = [&](typename Lds::Step& to, int t) {
#pragma unroll
    for (int i = 0; i < kMine; ++i) codes[i].unpack(to.tile[mine(i)], quarter);
    if (wave == 0) {
      // the first wave has the block's first row, whose window reaches back the furthest
      // (2048 rows after 16384 keys: one branch for the step's tiles 664 us, one
      // a tile 667, clearing without a branch 669)
      bool seen = true;   // all keys, as in most steps of a long sequence
#pragma unroll
      for (int u = 0; u < SUB; ++u) {
        const int tb = token(t + u);
        seen &= tb + kTile <= k.span.end && tb >= r.lo_min && ok[u] == 3u;
      }
      if (!seen) {
#pragma unroll
        for (int u = 0; u < SUB; ++u) words[u].clear_unseen(token(t + u), k.span.end, r.lo_min, a.sinks, ok[u]);
      }
      float top = 0.0f;
#pragma unroll
      for (int u = 0; u < SUB; ++u) top = fmaxf(top, words[u].largest_step());
      scale.see(top);
#pragma unroll
      for (int u = 0; u < SUB; ++u) words[u].put(to.tile[u].params, rf, scale.einv);
      if (lane == 0) {
        to.einv = scale.einv;
#pragma unroll
        for (int u = 0; u < SUB; ++u) to.ok[u] = ok[u];
      }
    }
  };
  if (k.t0 < k.t1) {
    fetch(k.t0);
    unpack(lds.step[0], k.t0);
    fetch(k.t0 + SUB);
    __syncthreads();
    int buffer = 0;
    for (int t = k.t0; t < k.t1; t += SUB, buffer ^= 1) {
      const typename Lds::Step& now = lds.step[buffer];
      int tb[SUB];
      bool seen = false;
#pragma unroll
      for (int u = 0; u < SUB; ++u) {
        tb[u] = t + u < k.t1 ? k.span.token(t + u) : 1 << 30;   // past the last tile: behind every row
        seen |= tile_seen(r, tb[u], a.sinks);
      }
      if (!idle && seen) {
        auto uniform = [](uint32_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)v); };
        w.set_scale(__uint_as_float(uniform(__float_as_uint(now.einv))));
        const uint32_t ok_now[SUB] = {uniform(now.ok[0]), uniform(now.ok[1])};
        const bool whole = !uneven && tile_whole(r, tb[0], k.sq.len, ok_now[0], a.sinks) &&
                           tile_whole(r, tb[1], k.sq.len, ok_now[1], a.sinks);
        w.template step<SUB>([&](int u, int s, int i) { return now.tile[u].k[s][i][lane]; },
                             [&](int u, int i) { return now.tile[u].v[i][lane]; },
                             [&](int u) -> const TileParams<D, G>& { return now.tile[u].params; }, tb, whole, k.sq.len,
                             ok_now, a.sinks);
      }
      unpack(lds.step[buffer ^ 1], t + SUB);
      fetch(t + 2 * SUB);
      __syncthreads();
    }
  }
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const float sum = w.finish(i);
    const int row = k.row0 + first + i * 16 + n;
    if (row >= k.rows) continue;
    if (k.active <= 1) {
      const int tok = row / a.heads_per_kv, h = k.hk * a.heads_per_kv + row - tok * a.heads_per_kv;
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;   // a row that sees nothing becomes 0
      const int64_t e = (int64_t)(k.sq.first + tok) * a.out.row_stride + (int64_t)h * a.out.head_stride + quad * 4;
#pragma unroll
      for (int d = 0; d < W::kTiles; ++d) store_out4(a.out, e + d * 16, w.o[i][d] * inv);
    } else {
      const int64_t at = part_index(a, k.b, k.hk, a.plan.row_blocks * Lds::kRows, row, k.split);
      if (quad == 0) {
        put_shared(a.part_ml + at * 2, w.maximum(i));
        put_shared(a.part_ml + at * 2 + 1, sum);
      }
#pragma unroll
      for (int d = 0; d < W::kTiles; ++d)
#pragma unroll
        for (int j = 0; j < 4; ++j) put_shared(a.part_o + at * D + d * 16 + quad * 4 + j, w.o[i][d][j]);
    }
  }
  if (k.active > 1) join_splits<D, NW * 64, 1>(a, k, Lds::kRows, reinterpret_cast<uint32_t*>(lds.top));
}

}  // namespace kv

namespace {

template <int V>
using IC = std::integral_constant<int, V>;

template <typename Lds>
hipError_t launch_attention(void (*kernel)(KvAttnArgs), int waves, const KvAttnArgs& a, hipStream_t st) {
  const unsigned blocks = (unsigned)((int64_t)a.c.kv_heads * a.b.seqs * a.plan.row_blocks * a.plan.splits);
  static_assert(sizeof(Lds) <= 160 * 1024, "LDS of a compute unit");
  if (sizeof(Lds) > 64 * 1024) {   // more than a launch gives without asking
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Lds));
    if (e != hipSuccess) return e;
  }
  KvAttnArgs args = a;
  void* ptrs[] = {&args};
  return hipLaunchKernel(reinterpret_cast<const void*>(kernel), dim3(blocks), dim3(waves * 64), ptrs,
                         sizeof(Lds), st);
}

// Every (row_tiles, waves) that the plan gives.
template <int BITS, int D, int G>
hipError_t with_plan(const KvAttnArgs& a, hipStream_t st) {
  const KvPlan& p = a.plan;
  auto few = [&](auto NT, auto NW) {
    return launch_attention<kv::FewLds<BITS, D, G, NT(), NW()>>(kv::k_kv_attention_few<BITS, D, G, NT(), NW()>, NW(), a, st);
  };
  if (p.row_waves == 1) {
    if constexpr (D <= 128) {
      if (p.row_tiles == 2) return p.key_waves == 8 ? few(IC<2>{}, IC<8>{}) : few(IC<2>{}, IC<4>{});
    }
    if constexpr (BITS * D <= 1024) {
      if (p.key_waves == 8) return few(IC<1>{}, IC<8>{});
    }
    return few(IC<1>{}, IC<4>{});
  }
  constexpr int NT = kv_many_tiles(D), NW = kv_many_waves(D);
  return launch_attention<kv::ManyLds<BITS, D, G, NT, NW>>(kv::k_kv_attention_many<BITS, D, G, NT, NW>, NW, a, st);
}

}  // namespace

template <int BITS, int D>
hipError_t run_kv_attention_form(const KvAttnArgs& a, hipStream_t st) {
  if (a.c.group == 32) return with_plan<BITS, D, 32>(a, st);
  if (a.c.group == 64) return with_plan<BITS, D, 64>(a, st);
  if constexpr (D >= 128) return with_plan<BITS, D, 128>(a, st);
  return hipErrorInvalidValue;   // refused before the launch
}

// This file is compiled once for every code width and head size.
template hipError_t run_kv_attention_form<ECHO_KV_BITS, ECHO_KV_HEAD_DIM>(const KvAttnArgs& a, hipStream_t st);

}  // namespace echo
