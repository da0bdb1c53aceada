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
// probabilities never leave their lane, and keys, values and parameters go
// from global memory to registers in the order the cache stores them
// (echo_kv_device.h): no LDS and no barrier in the loop.
//
// A wave works on NT tiles of 16 query rows (row = new token x query head of
// one K/V head) and walks 32 keys at a time, the next tile's loads in flight
// during the current one's arithmetic.  The running maximum moves only when a
// score exceeds it by more than 2^4, which keeps the rescaling of the output
// out of almost every step.
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

// What one step loads: keys and values of 2 x 16 tokens, and their parameters
// spread over the lanes (word 64 i + lane of [keys, values][half][token][group]).
// Every lane needs the parameters of 8 tokens, and loading them there would take
// 16 registers a group and buffer; they go through a few LDS words of the
// wave's own instead.
template <int BITS, int D, int G>
struct Tile {
  static constexpr int kRowBytes = D * BITS / 8;
  static constexpr int kKeyWords = kRowBytes / 16;       // words of a lane's share of one key row
  static constexpr int kUnitBytes = kRowBytes / 16;      // bytes of a lane's share of one value row
  static constexpr int kUnitWords = kUnitBytes < 4 ? 1 : kUnitBytes / 4;
  static constexpr int kGroups = D / G;
  uint32_t k[2][kKeyWords];
  uint32_t v[2][4][kUnitWords];
  static constexpr int kParamWords = 64 * kGroups;       // of a tile
  uint32_t param[kGroups];
  uint32_t ok;   // bit s: the 16 tokens of half s lie in a page of the cache
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
};
__device__ __forceinline__ Pages tile_pages(const KvCache& c, const int32_t* table, int len, int tb) {
  return Pages{{half_page(c, table, len, tb), half_page(c, table, len, tb + 16)}};
}

template <int BITS, int D, int G>
__device__ __forceinline__ void load_tile(Tile<BITS, D, G>& x, const KvCache& c, const Pages& pages,
                                          int hk, int tb) {
  using T = Tile<BITS, D, G>;
  const uint32_t n = threadIdx.x % 16, quad = threadIdx.x / 16 % 4;
  const uint32_t k_at = n * T::kRowBytes + quad * (T::kRowBytes / 4);
  const uint32_t v_at = quad * 4 * T::kRowBytes + n * T::kUnitBytes;
  const uint8_t* param[2][2];
  x.ok = 0;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    x.ok |= pages.p[s] < 0 ? 0u : 1u << s;
    const int64_t row = half_row(c, pages.p[s], hk, tb + 16 * s);
    const uint8_t* kc = c.k_codes + row * T::kRowBytes;
    const uint8_t* vc = c.v_codes + row * T::kRowBytes;
    param[0][s] = reinterpret_cast<const uint8_t*>(c.k_params + row * T::kGroups);
    param[1][s] = reinterpret_cast<const uint8_t*>(c.v_params + row * T::kGroups);
    load_words<T::kKeyWords>(kc + k_at, x.k[s]);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if constexpr (T::kUnitBytes == 2) x.v[s][r][0] = *reinterpret_cast<const uint16_t*>(vc + v_at + r * T::kRowBytes);
      else load_words<T::kUnitWords>(vc + v_at + r * T::kRowBytes, x.v[s][r]);
    }
  }
#pragma unroll
  for (int i = 0; i < T::kGroups; ++i) {
    const uint32_t w = i * 64 + threadIdx.x % 64;
    const uint32_t run = w / (16 * T::kGroups);          // 0, 1: keys of each half; 2, 3: values
    const uint8_t* lo = run & 1 ? param[0][1] : param[0][0];
    const uint8_t* hi = run & 1 ? param[1][1] : param[1][0];
    const uint8_t* p = run & 2 ? hi : lo;
    x.param[i] = *reinterpret_cast<const uint32_t*>(p + w % (16 * T::kGroups) * 4);
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

// Query rows of a block in LDS: their matrix operands, and what turns a raw
// score into log2 units.
template <int BITS, int D, int G, int ROWS>
struct QueryRows {
  static constexpr int kSlices = D / 32, kGroups = D / G, kRuns = D / 8;
  f16x8 op[ROWS / 16][kSlices][64];
  float rf[ROWS], qs[ROWS][kGroups];

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
    if (run % (G / 8) == 0) qs[r][run / (G / 8)] = sum * 0x1p-24f;
  }

  // Rows row0 .. row0 + ROWS - 1, each with its own power of two: the row's
  // largest element comes into [2^14, 2^15), and bf16 values keep all their
  // bits down to 2^-24 of the largest.
  template <int THREADS>
  __device__ __forceinline__ void stage(const KvAttnArgs& a, const Seq& sq, int hk, int row0, int rows) {
    static_assert(ROWS * kRuns % 64 == 0, "whole waves");
#pragma unroll
    for (int pass = 0; pass * THREADS < ROWS * kRuns; ++pass) {
      const int unit = pass * THREADS + threadIdx.x, r = unit / kRuns, run = unit % kRuns;
      if (unit >= ROWS * kRuns) break;
      float x[8], top = 0.0f;
      widen(load(a, sq, hk, row0 + r, rows, run), a.q.dtype, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(x[j]));
      top = run_reduce<kRuns>(top, [](float u, float v) { return fmaxf(u, v); });
      const int field = (int)(__float_as_uint(top) >> 23);
      const int up = field == 0 || field == 255 ? 0 : 14 - (field - 127);
      put(x, up, r, run);
      if (run == 0) rf[r] = ldexpf(a.scale_log2, 24 - up);
    }
  }

  // All rows with one power of two, from the largest finite element of the
  // block (a row 2^14 times smaller than another still keeps bf16's bits);
  // returns the factor from raw scores to log2 units.  top: a float per wave.
  template <int THREADS>
  __device__ __forceinline__ float stage_together(const KvAttnArgs& a, const Seq& sq, int hk, int row0, int rows,
                                                  float* tops) {
    constexpr int kPasses = ROWS * kRuns / THREADS;
    static_assert(ROWS * kRuns % THREADS == 0, "whole passes");
    u32x4 raw[kPasses];
#pragma unroll
    for (int pass = 0; pass < kPasses; ++pass) {
      const int unit = pass * THREADS + threadIdx.x;
      raw[pass] = load(a, sq, hk, row0 + unit / kRuns, rows, unit % kRuns);
    }
    float top = 0.0f;
#pragma unroll
    for (int pass = 0; pass < kPasses; ++pass) {
      float x[8];
      widen(raw[pass], a.q.dtype, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) top = fabsf(x[j]) < INFINITY ? fmaxf(top, fabsf(x[j])) : top;
    }
#pragma unroll
    for (int i = 1; i < 64; i *= 2) top = fmaxf(top, __shfl_xor(top, i));
    tops[threadIdx.x / 64] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < THREADS / 64; ++i) top = fmaxf(top, tops[i]);
    const int field = __builtin_amdgcn_readfirstlane((int)(__float_as_uint(top) >> 23));
    const int up = field == 0 ? 0 : 14 - (field - 127);
#pragma unroll
    for (int pass = 0; pass < kPasses; ++pass) {
      const int unit = pass * THREADS + threadIdx.x;
      float x[8];
      widen(raw[pass], a.q.dtype, x);
      put(x, up, unit / kRuns, unit % kRuns);
    }
    return ldexpf(a.scale_log2, 24 - up);
  }
};

// The state of a wave: 16 NT query rows against the keys seen so far.
template <int BITS, int D, int G, int NT>
struct Wave {
  static constexpr int kSlices = D / 32, kTiles = D / 16, kGroups = D / G;
  static constexpr float kHalf = BITS == 4 ? 8.0f : 128.0f;
  // Rows of `st`: g: sum p zero; kGroups + g: sum p step; 2 kGroups: sum p.
  // Eight groups leave no row for the last, which is added up in `l`.
  static constexpr bool kSumRow = 2 * kGroups < 16;
  f16x8 q[NT][kSlices];          // query rows as matrix operands, scaled to [2^14, 2^15)
  float qs[NT][kGroups];         // sum of a row's q over a group, * 2^-24
  float rf[NT];                  // raw score -> log2 units
  int lo[NT], hi[NT];            // visible keys: j <= hi and (j >= lo or j < sinks)
  f32x4 o[NT][kTiles];           // sum of p step einv (c - kHalf) 2^-9
  f32x4 st[NT];
  float l[NT];                   // (!kSumRow) this lane's part of sum p
  float mb[NT];                  // running maximum (log2) - kPeak
  float einv, elim;              // einv: a power of two with step einv <= 1 while every step <= elim
  uint32_t psel, por;            // how this lane builds its row of the operand that gives `st`
  int pgroup;

  // Rows row0 + first .. of the block's staged rows.
  template <int ROWS>
  __device__ __forceinline__ void begin(const KvAttnArgs& a, const Seq& sq, const QueryRows<BITS, D, G, ROWS>& from,
                                        int row0, int first, int rows) {
    const int n = threadIdx.x % 16, lane = threadIdx.x % 64;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int r = first + t * 16 + n, row = row0 + r;
      const bool exists = row < rows;
      const int pos = sq.len - sq.n + row / a.heads_per_kv;
      hi[t] = !a.causal || !exists ? sq.len - 1 : pos < sq.len ? pos : sq.len - 1;
      lo[t] = a.window > 0 && exists ? (int)max((int64_t)pos - a.window + 1, (int64_t)0) : 0;
      rf[t] = from.rf[r];
#pragma unroll
      for (int g = 0; g < kGroups; ++g) qs[t][g] = from.qs[r][g];
#pragma unroll
      for (int w = 0; w < kSlices; ++w) q[t][w] = from.op[first / 16 + t][w][lane];
      st[t] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < kTiles; ++i) o[t][i] = f32x4{0, 0, 0, 0};
      mb[t] = kLowest;
      l[t] = 0.0f;
    }
    einv = 1.0f;
    elim = 0.0f;
    psel = n < kGroups ? 0x07060302u : n < 2 * kGroups ? 0x05040100u : 0x0c0c0c0cu;
    por = n == 2 * kGroups ? 0x3c003c00u : 0u;
    pgroup = n % kGroups;
  }

  // One tile of 32 keys at token tb; masked: some of them some row may not see.
  // key(s, w): operand of slice w of half s; value(i): operand of value tile i;
  // param: the tile's parameters in LDS, 0 where there is no key; ok: as in Tile.
  template <typename Key, typename Value>
  __device__ __forceinline__ void step(const uint32_t* param, Key&& key, Value&& value, int tb, bool masked, int len,
                                       uint32_t ok, int sinks) {
    const int quad = threadIdx.x / 16 % 4;
    // words of tokens quad * 4 + 0..3 of half s, group minor
    auto params = [&](int array, int s, uint32_t (&w)[4][kGroups]) {
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        const u32x4 v = *reinterpret_cast<const u32x4*>(param + ((array * 2 + s) * 16 + quad * 4) * kGroups + 4 * i);
#pragma unroll
        for (int e = 0; e < 4; ++e) w[(4 * i + e) / kGroups][(4 * i + e) % kGroups] = v[e];
      }
    };
    float sc[NT][2][4];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      uint32_t kp[4][kGroups];
      params(0, s, kp);
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        f32x4 acc[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[t] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int w = g * G / 32; w < (g + 1) * G / 32; ++w) {
          const f16x8 a = key(s, w);
#pragma unroll
          for (int t = 0; t < NT; ++t) acc[t] = mfma(a, q[t][w], acc[t]);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float ks = f16_to_f32(kp[r][g] & 0xffffu), kz = f16_to_f32(kp[r][g] >> 16);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const float z = g == 0 ? kz * qs[t][g] : fmaf(kz, qs[t][g], sc[t][s][r]);
            sc[t][s][r] = fmaf(ks, acc[t][r], z);
          }
        }
      }
    }
    if (masked) {
      int from = tb;
      asm volatile("" : "+s"(from));   // the comparisons stay in this branch
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int j = from + 16 * s + quad * 4 + r;
          const bool there = j < len && (ok >> s & 1u);
#pragma unroll
          for (int t = 0; t < NT; ++t)
            if (!(there && j <= hi[t] && (j >= lo[t] || j < sinks))) sc[t][s][r] = rf[t] < 0.0f ? INFINITY : -INFINITY;
        }
    }
    float y[NT][2][4], vs[2][4][kGroups];
    uint32_t vp[2][4][kGroups];
    float top_y = -INFINITY, top_step = 0.0f;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      params(1, s, vp[s]);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          vs[s][r][g] = f16_to_f32(vp[s][r][g] & 0xffffu);
          top_step = fmaxf(top_step, vs[s][r][g]);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          y[t][s][r] = fmaf(sc[t][s][r], rf[t], -mb[t]);
          top_y = fmaxf(top_y, y[t][s][r]);
        }
      }
    }
    if (__any(top_y > kPeak + kSlack || top_step > elim)) {
      rescale(sc, top_step);
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int r = 0; r < 4; ++r) y[t][s][r] = fmaf(sc[t][s][r], rf[t], -mb[t]);
    }
    // the operand of the sums that need no code: zeros, steps, ones
    uint32_t sw[2][4];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if constexpr (kGroups == 1) sw[s][r] = vp[s][r][0];
        else sw[s][r] = param[((2 + s) * 16 + quad * 4 + r) * kGroups + pgroup];
      }
    auto pick = [&](int s, int r) { return __builtin_amdgcn_perm(sw[s][r + 1], sw[s][r], psel) | por; };
    const f16x8 sums = operand(pick(0, 0), pick(0, 2), pick(1, 0), pick(1, 2));
    f16x8 pv[NT][kGroups];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int g = 0; g < kGroups; ++g) vs[s][r][g] *= einv;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      f16x8 p;
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float e = __builtin_amdgcn_exp2f(y[t][s][r]);
          p[4 * s + r] = (_Float16)e;
          if constexpr (!kSumRow) l[t] += e;
#pragma unroll
          for (int g = 0; g < kGroups; ++g) pv[t][g][4 * s + r] = (_Float16)(e * vs[s][r][g]);
        }
      st[t] = mfma(sums, p, st[t]);
    }
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      const f16x8 a = value(i);
#pragma unroll
      for (int t = 0; t < NT; ++t) o[t][i] = mfma(a, pv[t][i * 16 / G], o[t][i]);
    }
  }

  // Raise the running maxima to the largest scores and the normaliser to the largest step.
  __device__ __forceinline__ void rescale(const float (&sc)[NT][2][4], float top_step) {
    top_step = fmaxf(top_step, __shfl_xor(top_step, 16));
    top_step = fmaxf(top_step, __shfl_xor(top_step, 32));
    float ratio = 1.0f;
    if (top_step > elim) {      // the same in the whole wave
      const int e = (int)(__float_as_uint(top_step) >> 23) - 127 + 1;   // top_step 2^-e in [1/2, 1)
      const float inv = ldexpf(1.0f, -e);
      ratio = elim > 0.0f ? inv / einv : 1.0f;   // powers of two
      einv = inv;
      elim = ldexpf(1.0f, e);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float top = mb[t] + kPeak;
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int r = 0; r < 4; ++r) top = fmaxf(top, sc[t][s][r] * rf[t]);
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      top -= kPeak;
      const float alpha = __builtin_amdgcn_exp2f(mb[t] - top);
      mb[t] = top;
      st[t] *= alpha;
      l[t] *= alpha;
      const float both = alpha * ratio;
#pragma unroll
      for (int i = 0; i < kTiles; ++i) o[t][i] *= both;
    }
  }

  // Row `row` of the sums' result for this lane's query row, from the lane that holds it.
  __device__ __forceinline__ float sum_of(int t, int row) const {
    return __shfl(st[t][row % 4], (int)(threadIdx.x % 16) + 16 * (row / 4));
  }

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
    if constexpr (kSumRow) return sum_of(t, 2 * kGroups);
    float sum = l[t] + __shfl_xor(l[t], 16);
    return sum + __shfl_xor(sum, 32);
  }
};

// What a block works on, and the bounds over a range of its rows: a tile inside
// all of them needs no mask, one outside all of them nothing.
struct Block {
  Seq sq;
  Span span;
  int b, hk, split, row0, rows, active, t0, t1;
  const int32_t* table;
};
struct Bounds {
  int hi_min, hi_max, lo_min, lo_max;
};

// grid.x: K/V head fastest, then split, then block of rows (the last rows
// first: under a causal mask they have the most keys); grid.y: sequence.
// False: the block has nothing to do.
__device__ __forceinline__ bool block_of(const KvAttnArgs& a, int block_rows, Block& k) {
  k.b = blockIdx.y;
  k.hk = blockIdx.x % a.c.kv_heads;
  const int rest = blockIdx.x / a.c.kv_heads;
  k.split = rest % a.plan.splits;
  k.sq = sequence(a, k.b);
  k.rows = k.sq.computed * a.heads_per_kv;
  k.row0 = (a.plan.row_blocks - 1 - rest / a.plan.splits) * block_rows;
  if (k.row0 >= k.rows) return false;
  const int last = min(k.row0 + block_rows, k.rows) - 1;
  k.span = key_span(a, k.sq.len, k.sq.n, k.row0 / a.heads_per_kv, last / a.heads_per_kv);
  k.active = (k.span.tiles + a.plan.split_tiles - 1) / a.plan.split_tiles;
  k.t0 = k.split * a.plan.split_tiles;
  k.t1 = min(k.t0 + a.plan.split_tiles, k.span.tiles);
  k.table = a.b.page_table + (int64_t)k.b * a.b.table_stride;
  return k.split == 0 || k.split < k.active;
}
__device__ __forceinline__ Bounds bounds_of(const KvAttnArgs& a, const Block& k, int first, int last) {
  const int p0 = k.sq.len - k.sq.n + first / a.heads_per_kv, p1 = k.sq.len - k.sq.n + last / a.heads_per_kv;
  return Bounds{a.causal ? p0 : k.sq.len - 1, a.causal ? p1 : k.sq.len - 1,
                a.window > 0 ? p0 - a.window + 1 : 0, a.window > 0 ? p1 - a.window + 1 : 0};
}
__device__ __forceinline__ bool tile_seen(const Bounds& r, int tb, int sinks) {
  return tb <= r.hi_max && (tb + kTile > r.lo_min || tb < sinks);
}
__device__ __forceinline__ bool tile_whole(const Bounds& r, int tb, int len, uint32_t ok, int sinks) {
  return tb + kTile - 1 <= r.hi_min && tb + kTile <= len && ok == 3u && (tb >= r.lo_max || tb + kTile <= sinks);
}

// A word of the tile's parameters, 0 for a token that is not there (its slot may hold anything).
template <int GROUPS>
__device__ __forceinline__ uint32_t there_or_zero(uint32_t word, int w, int tb, int len, uint32_t ok) {
  const int s = w / (16 * GROUPS) & 1, j = tb + 16 * s + w % (16 * GROUPS) / GROUPS;
  return j < len && (ok >> s & 1u) ? word : 0u;
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

// ------------------------------------------------------------------ few rows
// The NW waves of a block share its 16 NT rows and take turns over the keys:
// wave w has the tiles w, w + NW, ...  Loads go to registers, the next tile's
// in flight during the current one's arithmetic; no barrier in the loop.  At
// the end the waves' results meet in LDS.
template <int BITS, int D, int G, int NT, int NW>
struct FewLds {
  static constexpr int kRows = NT * 16, kStride = D + 4;
  QueryRows<BITS, D, G, kRows> q;
  uint32_t param[NW][Tile<BITS, D, G>::kParamWords];
  float m[NW][kRows], l[NW][kRows];
  float o[NW][kRows][kStride];
};

// Waves per SIMD that the registers have to leave room for.
constexpr int few_min_waves(int D, int NT) {
  return NT == 1 ? (D == 64 ? 4 : D == 128 ? 3 : 2) : NT == 2 && D <= 128 ? 2 : 1;
}

template <int BITS, int D, int G, int NT, int NW>
__global__ __launch_bounds__(NW * 64, few_min_waves(D, NT)) void k_kv_attention_few(KvAttnArgs a) {
  using W = Wave<BITS, D, G, NT>;
  using Lds = FewLds<BITS, D, G, NT, NW>;
  extern __shared__ __align__(16) uint8_t shared[];
  Lds& lds = *reinterpret_cast<Lds*>(shared);
  Block k;
  if (!block_of(a, Lds::kRows, k)) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  int t = k.t0 + wave;
  Tile<BITS, D, G> x, y;
  Pages next = {{-1, -1}};
  // a load past the last tile repeats it; nothing uses the copy
  auto fetch = [&](Tile<BITS, D, G>& into, int at) {
    load_tile(into, a.c, next, k.hk, k.span.token(min(at, k.t1 - 1)));
    next = tile_pages(a.c, k.table, k.sq.len, k.span.token(min(at + NW, k.t1 - 1)));
  };
  if (t < k.t1) {
    next = tile_pages(a.c, k.table, k.sq.len, k.span.token(t));
    fetch(x, t);
  }
  lds.q.template stage<NW * 64>(a, k.sq, k.hk, k.row0, k.rows);
  __syncthreads();
  W w;
  w.begin(a, k.sq, lds.q, k.row0, 0, k.rows);
  const Bounds r = bounds_of(a, k, k.row0, min(k.row0 + Lds::kRows, k.rows) - 1);
  uint32_t* param = lds.param[wave];
  for (; t < k.t1; t += NW) {
    fetch(y, t + NW);
    const int tb = k.span.token(t);
    if (tile_seen(r, tb, a.sinks)) {
      const bool whole = tile_whole(r, tb, k.sq.len, x.ok, a.sinks);
      wave_sync();
#pragma unroll
      for (int i = 0; i < W::kGroups; ++i) {
        const int at = i * 64 + threadIdx.x % 64;
        param[at] = whole ? x.param[i] : there_or_zero<W::kGroups>(x.param[i], at, tb, k.sq.len, x.ok);
      }
      wave_sync();
      w.step(param, [&](int s, int i) { return key_operand<BITS>(x.k[s], i); },
             [&](int i) { return value_operand<BITS>(x.v, i); }, tb, !whole, k.sq.len, x.ok, a.sinks);
    }
    x = y;
  }
  const int n = threadIdx.x % 16, quad = threadIdx.x / 16 % 4;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const float l = w.finish(i);
    const int row = i * 16 + n;
    if (quad == 0) {
      lds.m[wave][row] = w.mb[i];
      lds.l[wave][row] = l;
    }
#pragma unroll
    for (int e = 0; e < W::kTiles; ++e) *reinterpret_cast<f32x4*>(&lds.o[wave][row][e * 16 + quad * 4]) = w.o[i][e];
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
      for (int e = 0; e < 8; ++e) v[e] = fmaf(lds.o[i][r0][run * 8 + e], f, v[e]);
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
        a.part_ml[at * 2] = top;
        a.part_ml[at * 2 + 1] = sum;
      }
      f32x4* to = reinterpret_cast<f32x4*>(a.part_o + at * D + run * 8);
      to[0] = f32x4{v[0], v[1], v[2], v[3]};
      to[1] = f32x4{v[4], v[5], v[6], v[7]};
    }
  }
}

// ------------------------------------------------------------------ many rows
// Each of the NW waves of a block has its own 16 NT rows and all walk the same
// keys, two tiles of 32 a step.  The waves unpack the codes once, each a quarter
// of one tile, into matrix operands in LDS (two buffers, one barrier a step),
// and one wave the parameters into what the softmax uses; doing either per wave
// would cost as much as the softmax.  The block's query rows share one power of
// two, so that a score in log2 units less the running maximum takes two
// multiply-adds: a key's step and the row factor are one number.
template <int BITS, int D, int G>
struct ManyTile {
  static constexpr int kGroups = D / G;
  f16x8 k[2][D / 32][64];
  f16x8 v[D / 16][64];
  f16x8 sums[64];                       // rows: zeros, steps, ones (see Wave::st)
  float kstep[2][16][kGroups];          // key step * row factor
  float kzero[2][16][kGroups];
  float vstep[2][16][kGroups];          // value step * einv
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
  float top[NW];
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

// A tile's parameters in one wave's registers.
template <int BITS, int D, int G>
struct TileParams {
  using T = Tile<BITS, D, G>;
  uint32_t param[T::kGroups];
  uint32_t ok;

  __device__ __forceinline__ void load(const KvCache& c, const int32_t* table, int len, int hk, int tb) {
    int64_t row[2];
    ok = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int page = half_page(c, table, len, tb + 16 * i);
      ok |= page < 0 ? 0u : 1u << i;
      row[i] = half_row(c, page, hk, tb + 16 * i);
    }
#pragma unroll
    for (int i = 0; i < T::kGroups; ++i) {
      const uint32_t w = i * 64 + threadIdx.x % 64, run = w / (16 * T::kGroups);
      const uint32_t* from = run & 2 ? c.v_params : c.k_params;
      param[i] = from[(run & 1 ? row[1] : row[0]) * T::kGroups + w % (16 * T::kGroups)];
    }
  }
  // Parameters of tokens that are not there become 0: their slots may hold anything.
  __device__ __forceinline__ void clear_missing(int tb, int len) {
#pragma unroll
    for (int i = 0; i < T::kGroups; ++i) param[i] = there_or_zero<T::kGroups>(param[i], i * 64 + threadIdx.x % 64, tb, len, ok);
  }
  __device__ __forceinline__ float largest_step() const {   // of this lane's values
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < T::kGroups; ++i)
      if (i * 64 + threadIdx.x % 64 >= 32 * T::kGroups) top = fmaxf(top, f16_to_f32(param[i] & 0xffffu));
    return top;
  }
  __device__ __forceinline__ void unpack_params(ManyTile<BITS, D, G>& to, float rf, float einv) const {
#pragma unroll
    for (int i = 0; i < T::kGroups; ++i) {
      const int w = i * 64 + threadIdx.x % 64, at = w % (32 * T::kGroups);   // [half][token][group]
      const float step = f16_to_f32(param[i] & 0xffffu);
      if (w < 32 * T::kGroups) {
        (&to.kstep[0][0][0])[at] = step * rf;
        (&to.kzero[0][0][0])[at] = f16_to_f32(param[i] >> 16);
      } else {
        (&to.vstep[0][0][0])[at] = step * einv;
        const int g = at % T::kGroups, token = at / T::kGroups, j = token / 16 * 4 + token % 4;
        uint16_t* zeros = reinterpret_cast<uint16_t*>(&to.sums[token % 16 / 4 * 16 + g]);
        uint16_t* steps = reinterpret_cast<uint16_t*>(&to.sums[token % 16 / 4 * 16 + T::kGroups + g]);
        zeros[j] = (uint16_t)(param[i] >> 16);
        steps[j] = (uint16_t)param[i];
      }
    }
  }
};

template <int BITS, int D, int G, int NT, int NW>
__global__ __launch_bounds__(NW * 64, D == 64 ? 3 : 2) void k_kv_attention_many(KvAttnArgs a) {
  using Lds = ManyLds<BITS, D, G, NT, NW>;
  using MT = ManyTile<BITS, D, G>;
  constexpr int kSlices = D / 32, kTiles = D / 16, kGroups = D / G, SUB = kSub;
  constexpr float kHalf = BITS == 4 ? 8.0f : 128.0f;
  constexpr bool kSumRow = 2 * kGroups < 16;   // see Wave
  extern __shared__ __align__(16) uint8_t shared[];
  Lds& lds = *reinterpret_cast<Lds*>(shared);
  Block k;
  if (!block_of(a, Lds::kRows, k)) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int lane = threadIdx.x % 64, n = lane % 16, quad = lane / 16;
  const int first = wave * NT * 16;

  const float rf = lds.q.template stage_together<NW * 64>(a, k.sq, k.hk, k.row0, k.rows, lds.top);
  __syncthreads();
  f16x8 q[NT][kSlices];
  float qs[NT][kGroups], mb[NT], l[NT];
  int lo[NT], hi[NT];
  f32x4 o[NT][kTiles], st[NT];
  bool none[NT];               // no key seen yet
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int r = first + t * 16 + n, row = k.row0 + r;
    const bool exists = row < k.rows;
    const int pos = k.sq.len - k.sq.n + row / a.heads_per_kv;
    hi[t] = !a.causal || !exists ? k.sq.len - 1 : pos < k.sq.len ? pos : k.sq.len - 1;
    lo[t] = a.window > 0 && exists ? (int)max((int64_t)pos - a.window + 1, (int64_t)0) : 0;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) qs[t][g] = lds.q.qs[r][g] * rf;
#pragma unroll
    for (int w = 0; w < kSlices; ++w) q[t][w] = lds.q.op[first / 16 + t][w][lane];
    st[t] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kTiles; ++i) o[t][i] = f32x4{0, 0, 0, 0};
    mb[t] = 0.0f;
    l[t] = 0.0f;
    none[t] = true;
  }
  bool fresh = true;           // some row of the wave has seen no key yet
  float einv = 1.0f;           // of this wave's o
  __syncthreads();             // the steps overwrite the staged rows
  // what no step writes: the row of ones, and rows of zeros behind it
  for (int i = threadIdx.x; i < 2 * SUB * 64; i += NW * 64) {
    const uint32_t one = kSumRow && i % 16 == 2 * kGroups ? 0x3c003c00u : 0u;
    lds.step[i / (SUB * 64)].tile[i / 64 % SUB].sums[i % 64] = operand(one, one, one, one);
  }
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
  TileParams<BITS, D, G> params[SUB];
  float next_einv = 1.0f, limit = 0.0f;          // first wave: what the coming step's values are scaled by
  auto token = [&](int t) { return k.span.token(min(t, k.t1 - 1)); };   // past the last tile: that one again
  auto fetch = [&](int t) {
#pragma unroll
    for (int i = 0; i < kMine; ++i) codes[i].load(a.c, k.table, k.sq.len, k.hk, token(t + mine(i)), quarter);
    if (wave == 0) {
#pragma unroll
      for (int u = 0; u < SUB; ++u) params[u].load(a.c, k.table, k.sq.len, k.hk, token(t + u));
    }
  };
  auto unpack = [&](typename Lds::Step& to, int t) {
#pragma unroll
    for (int i = 0; i < kMine; ++i) codes[i].unpack(to.tile[mine(i)], quarter);
    if (wave == 0) {
      float top = 0.0f;
#pragma unroll
      for (int u = 0; u < SUB; ++u) {
        params[u].clear_missing(token(t + u), k.sq.len);
        top = fmaxf(top, params[u].largest_step());
      }
      if (__any(top > limit)) {   // rare: products of probability and step stay in f16's range
#pragma unroll
        for (int i = 1; i < 64; i *= 2) top = fmaxf(top, __shfl_xor(top, i));
        const int e = (int)(__float_as_uint(top) >> 23) - 127 + 1;   // top 2^-e in [1/2, 1)
        next_einv = ldexpf(1.0f, -e);
        limit = ldexpf(1.0f, e);
      }
#pragma unroll
      for (int u = 0; u < SUB; ++u) params[u].unpack_params(to.tile[u], rf, next_einv);
      if (lane == 0) {
        to.einv = next_einv;
#pragma unroll
        for (int u = 0; u < SUB; ++u) to.ok[u] = params[u].ok;
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
        const float e = __uint_as_float(uniform(__float_as_uint(now.einv)));
        const uint32_t ok_now[SUB] = {uniform(now.ok[0]), uniform(now.ok[1])};
        const bool whole = tile_whole(r, tb[0], k.sq.len, ok_now[0], a.sinks) &&
                           tile_whole(r, tb[1], k.sq.len, ok_now[1], a.sinks);
        if (e != einv) {
          const float ratio = e / einv;   // powers of two
#pragma unroll
          for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < kTiles; ++j) o[i][j] *= ratio;
          einv = e;
        }
        // scores, in log2 units less the running maximum
        float y[SUB][NT][2][4];
#pragma unroll
        for (int u = 0; u < SUB; ++u) {
          const MT& x = now.tile[u];
#pragma unroll
          for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
              f32x4 acc[NT];
#pragma unroll
              for (int i = 0; i < NT; ++i) acc[i] = f32x4{0, 0, 0, 0};
#pragma unroll
              for (int w = g * G / 32; w < (g + 1) * G / 32; ++w) {
                const f16x8 op = x.k[s][w][lane];
#pragma unroll
                for (int i = 0; i < NT; ++i) acc[i] = mfma(op, q[i][w], acc[i]);
              }
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float ks = x.kstep[s][quad * 4 + j][g], kz = x.kzero[s][quad * 4 + j][g];
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                  const float z = fmaf(kz, qs[i][g], g == 0 ? -mb[i] : y[u][i][s][j]);
                  y[u][i][s][j] = fmaf(ks, acc[i][j], z);
                }
              }
            }
          }
        }
        if (!whole) {
#pragma unroll
          for (int u = 0; u < SUB; ++u)
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const int key = tb[u] + 16 * s + quad * 4 + j;
                const bool there = key < k.sq.len && (ok_now[u] >> s & 1u);
#pragma unroll
                for (int i = 0; i < NT; ++i)
                  if (!(there && key <= hi[i] && (key >= lo[i] || key < a.sinks))) y[u][i][s][j] = -INFINITY;
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
            const float up = !any ? 0.0f : none[i] ? m - kPeak : fmaxf(m - kPeak, 0.0f);
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
#pragma unroll
        for (int u = 0; u < SUB; ++u) {
          const MT& x = now.tile[u];
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
                if constexpr (!kSumRow) l[i] += e;
#pragma unroll
                for (int g = 0; g < kGroups; ++g) pv[i][g][4 * s + j] = (_Float16)(e * x.vstep[s][quad * 4 + j][g]);
              }
            st[i] = mfma(sums, p, st[i]);
          }
#pragma unroll
          for (int d = 0; d < kTiles; ++d) {
            const f16x8 op = x.v[d][lane];
#pragma unroll
            for (int i = 0; i < NT; ++i) o[i][d] = mfma(op, pv[i][d * 16 / G], o[i][d]);
          }
        }
      }
      unpack(lds.step[buffer ^ 1], t + SUB);
      fetch(t + 2 * SUB);
      __syncthreads();
    }
  }
  auto sum_of = [&](int i, int row) { return __shfl(st[i][row % 4], n + 16 * (row / 4)); };
  const float up = 0x1p9f / einv;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const float z = fmaf(kHalf, sum_of(i, kGroups + g), sum_of(i, g));
#pragma unroll
      for (int d = g * G / 16; d < (g + 1) * G / 16; ++d)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][d][j] = fmaf(o[i][d][j], up, z);
    }
    float sum;
    if constexpr (kSumRow) {
      sum = sum_of(i, 2 * kGroups);
    } else {
      sum = l[i] + __shfl_xor(l[i], 16);
      sum += __shfl_xor(sum, 32);
    }
    const int row = k.row0 + first + i * 16 + n;
    if (row >= k.rows) continue;
    if (k.active <= 1) {
      const int tok = row / a.heads_per_kv, h = k.hk * a.heads_per_kv + row - tok * a.heads_per_kv;
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;   // a row that sees nothing becomes 0
      const int64_t e = (int64_t)(k.sq.first + tok) * a.out.row_stride + (int64_t)h * a.out.head_stride + quad * 4;
#pragma unroll
      for (int d = 0; d < kTiles; ++d) store_out4(a.out, e + d * 16, o[i][d] * inv);
    } else {
      const int64_t at = part_index(a, k.b, k.hk, a.plan.row_blocks * Lds::kRows, row, k.split);
      if (quad == 0) {
        a.part_ml[at * 2] = none[i] ? kLowest : mb[i];
        a.part_ml[at * 2 + 1] = sum;
      }
#pragma unroll
      for (int d = 0; d < kTiles; ++d) *reinterpret_cast<f32x4*>(a.part_o + at * D + d * 16 + quad * 4) = o[i][d];
    }
  }
}

}  // namespace kv

namespace {

template <int V>
using IC = std::integral_constant<int, V>;

template <typename Lds>
hipError_t launch_attention(void (*kernel)(KvAttnArgs), int waves, const KvAttnArgs& a, hipStream_t st) {
  const unsigned blocks = (unsigned)((int64_t)a.c.kv_heads * a.plan.row_blocks * a.plan.splits);
  static_assert(sizeof(Lds) <= 160 * 1024, "LDS of a compute unit");
  if (sizeof(Lds) > 64 * 1024) {   // more than a launch gives without asking
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Lds));
    if (e != hipSuccess) return e;
  }
  KvAttnArgs args = a;
  void* ptrs[] = {&args};
  return hipLaunchKernel(reinterpret_cast<const void*>(kernel), dim3(blocks, a.b.seqs), dim3(waves * 64), ptrs,
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
    if (p.row_tiles == 1 && p.key_waves == 4) return few(IC<1>{}, IC<4>{});
    if (p.row_tiles == 1) return few(IC<1>{}, IC<8>{});
    if (p.row_tiles == 2) return few(IC<2>{}, IC<4>{});
    if constexpr (D <= 128) {
      if (p.row_tiles == 3) return few(IC<3>{}, IC<4>{});
    }
    return hipErrorInvalidValue;
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
