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

// What one step loads: keys and values of 2 x 16 tokens and their parameters.
template <int BITS, int D, int G>
struct Tile {
  static constexpr int kRowBytes = D * BITS / 8;
  static constexpr int kKeyWords = kRowBytes / 16;       // words of a lane's share of one key row
  static constexpr int kUnitBytes = kRowBytes / 16;      // bytes of a lane's share of one value row
  static constexpr int kUnitWords = kUnitBytes < 4 ? 1 : kUnitBytes / 4;
  static constexpr int kGroups = D / G;
  uint32_t k[2][kKeyWords];
  uint32_t v[2][4][kUnitWords];
  uint32_t kp[2][4][kGroups], vp[2][4][kGroups];
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

// Pages of the two halves of the tile at token tb, -1 where there is none: the
// same in all lanes, so they are scalar loads.
struct Pages {
  int p[2];
};
__device__ __forceinline__ Pages tile_pages(const KvCache& c, const int32_t* table, int len, int tb) {
  typedef const int32_t __attribute__((address_space(4))) * scalar_ptr;
  Pages r;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int t = tb + 16 * s;
    int page = -1;
    if (t < len) page = ((scalar_ptr)(uintptr_t)table)[t >> c.page_shift];
    r.p[s] = page >= 0 && page < c.num_pages ? page : -1;
  }
  return r;
}

template <int BITS, int D, int G>
__device__ __forceinline__ void load_tile(Tile<BITS, D, G>& x, const KvCache& c, const Pages& pages,
                                          int hk, int tb) {
  using T = Tile<BITS, D, G>;
  const uint32_t n = threadIdx.x % 16, quad = threadIdx.x / 16 % 4;
  const uint32_t k_at = n * T::kRowBytes + quad * (T::kRowBytes / 4);
  const uint32_t v_at = quad * 4 * T::kRowBytes + n * T::kUnitBytes;
  const uint32_t p_at = quad * 16 * T::kGroups;
  x.ok = 0;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    // a half without a page reads page 0, whose memory exists, and is masked
    const int64_t page = pages.p[s] < 0 ? 0 : pages.p[s];
    x.ok |= pages.p[s] < 0 ? 0u : 1u << s;
    const int64_t row = ((page * c.kv_heads + hk) << c.page_shift) + ((tb + 16 * s) & ((1 << c.page_shift) - 1));
    const uint8_t* kc = c.k_codes + row * T::kRowBytes;
    const uint8_t* vc = c.v_codes + row * T::kRowBytes;
    const uint8_t* kp = reinterpret_cast<const uint8_t*>(c.k_params) + row * (4 * T::kGroups);
    const uint8_t* vp = reinterpret_cast<const uint8_t*>(c.v_params) + row * (4 * T::kGroups);
    load_words<T::kKeyWords>(kc + k_at, x.k[s]);
    load_words<4 * T::kGroups>(kp + p_at, &x.kp[s][0][0]);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if constexpr (T::kUnitBytes == 2) x.v[s][r][0] = *reinterpret_cast<const uint16_t*>(vc + v_at + r * T::kRowBytes);
      else load_words<T::kUnitWords>(vc + v_at + r * T::kRowBytes, x.v[s][r]);
    }
    load_words<4 * T::kGroups>(vp + p_at, &x.vp[s][0][0]);
  }
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

// The state of a wave: 16 NT query rows against the keys seen so far.
template <int BITS, int D, int G, int NT>
struct Wave {
  static constexpr int kSlices = D / 32, kTiles = D / 16, kGroups = D / G;
  static constexpr float kHalf = BITS == 4 ? 8.0f : 128.0f;
  f16x8 q[NT][kSlices];          // query rows as matrix operands, scaled to [2^14, 2^15)
  float qs[NT][kGroups];         // sum of a row's q over a group, * 2^-24
  float rf[NT];                  // raw score -> log2 units
  int lo[NT], hi[NT];            // visible keys: j <= hi and (j >= lo or j < sinks)
  f32x4 o[NT][kTiles];           // sum of p step einv (c - kHalf) 2^-9
  // Rows of a 16x16 result: g: sum p zero; kGroups + g: sum p step; 2 kGroups:
  // sum p.  Eight groups leave no row for the last, which is added up in `l`.
  static constexpr bool kSumRow = 2 * kGroups < 16;
  f32x4 st[NT];
  float l[NT];                   // (!kSumRow) this lane's part of sum p
  float mb[NT];                  // running maximum (log2) - kPeak
  float einv, elim;              // einv: a power of two with step einv <= 1 while every step <= elim
  uint32_t psel, por;            // how this lane builds its row of the operand that gives `st`
  int pgroup;

  // The rows base .. base + 16 NT - 1 of a (sequence, K/V head) with `rows` rows.
  __device__ __forceinline__ void begin(const KvAttnArgs& a, const Seq& sq, int hk, int base, int rows) {
    const int n = threadIdx.x % 16, quad = threadIdx.x / 16 % 4;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int row = base + t * 16 + n;
      const bool exists = row < rows;
      const int i = row / a.heads_per_kv, h = row - i * a.heads_per_kv;
      const int pos = sq.len - sq.n + i;
      hi[t] = !a.causal || !exists ? sq.len - 1 : pos < sq.len ? pos : sq.len - 1;
      lo[t] = a.window > 0 && exists ? (int)max((int64_t)pos - a.window + 1, (int64_t)0) : 0;
      const uint16_t* src = static_cast<const uint16_t*>(a.q.p) + (int64_t)(sq.first + (exists ? i : 0)) * a.q.row_stride +
                            (int64_t)(hk * a.heads_per_kv + (exists ? h : 0)) * a.q.head_stride + quad * 8;
      u32x4 raw[kSlices];
#pragma unroll
      for (int w = 0; w < kSlices; ++w) raw[w] = *reinterpret_cast<const u32x4*>(src + w * 32);
      auto value = [&](int w, int j) {
        const uint32_t bits = j & 1 ? raw[w][j / 2] >> 16 : raw[w][j / 2] & 0xffffu;
        return exists ? (a.q.dtype == kKvF16 ? f16_to_f32(bits) : bf16_to_f32(bits)) : 0.0f;
      };
      float top = 0.0f;
#pragma unroll
      for (int w = 0; w < kSlices; ++w)
#pragma unroll
        for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(value(w, j)));
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      // a power of two takes the row's largest element into [2^14, 2^15): bf16
      // values keep all their bits down to 2^-24 of the largest
      const int field = (int)(__float_as_uint(top) >> 23);
      const int up = field == 0 || field == 255 ? 0 : 14 - (field - 127);
      rf[t] = ldexpf(a.scale_log2, 24 - up);
#pragma unroll
      for (int g = 0; g < kGroups; ++g) qs[t][g] = 0.0f;
#pragma unroll
      for (int w = 0; w < kSlices; ++w) {
        _Float16 e[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float x = ldexpf(value(w, j), up);
          e[j] = (_Float16)x;
          qs[t][w * 32 / G] += (float)e[j];
        }
        f16x8 op;
        const _Float16 low = (_Float16)0.0625f;
        if constexpr (BITS == 4) {
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            op[2 * v] = v & 1 ? e[v] * low : e[v];
            op[2 * v + 1] = v & 1 ? e[v + 4] * low : e[v + 4];
          }
        } else {
          op = f16x8{e[0], e[2], e[1], e[3], e[4], e[6], e[5], e[7]};
        }
        q[t][w] = op;
      }
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        qs[t][g] += __shfl_xor(qs[t][g], 16);
        qs[t][g] += __shfl_xor(qs[t][g], 32);
        qs[t][g] *= 0x1p-24f;
      }
      st[t] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int i2 = 0; i2 < kTiles; ++i2) o[t][i2] = f32x4{0, 0, 0, 0};
      mb[t] = kLowest;
      l[t] = 0.0f;
    }
    einv = 1.0f;
    elim = 0.0f;
    psel = n < kGroups ? 0x07060302u : n < 2 * kGroups ? 0x05040100u : 0x0c0c0c0cu;
    por = n == 2 * kGroups ? 0x3c003c00u : 0u;
    pgroup = n < kGroups ? n : n - kGroups;
  }

  // One tile of 32 keys at token tb; masked: some of them some row may not see.
  __device__ __forceinline__ void step(Tile<BITS, D, G>& x, int tb, bool masked, int len, int sinks) {
    const int quad = threadIdx.x / 16 % 4;
    float sc[NT][2][4];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        f32x4 acc[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[t] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int w = g * G / 32; w < (g + 1) * G / 32; ++w) {
          const f16x8 a = key_operand<BITS>(x.k[s], w);
#pragma unroll
          for (int t = 0; t < NT; ++t) acc[t] = mfma(a, q[t][w], acc[t]);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float ks = f16_to_f32(x.kp[s][r][g] & 0xffffu), kz = f16_to_f32(x.kp[s][r][g] >> 16);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const float z = g == 0 ? kz * qs[t][g] : fmaf(kz, qs[t][g], sc[t][s][r]);
            sc[t][s][r] = fmaf(ks, acc[t][r], z);
          }
        }
      }
    }
    if (masked) {
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int j = tb + 16 * s + quad * 4 + r;
          const bool there = j < len && (x.ok >> s & 1u);
#pragma unroll
          for (int g = 0; g < kGroups; ++g)
            if (!there) x.vp[s][r][g] = 0u;   // slots behind the last key hold anything
#pragma unroll
          for (int t = 0; t < NT; ++t)
            if (!(there && j <= hi[t] && (j >= lo[t] || j < sinks))) sc[t][s][r] = rf[t] < 0.0f ? INFINITY : -INFINITY;
        }
    }
    float y[NT][2][4], vs[2][4][kGroups];
    float top_y = -INFINITY, top_step = 0.0f;
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          vs[s][r][g] = f16_to_f32(x.vp[s][r][g] & 0xffffu);
          top_step = fmaxf(top_step, vs[s][r][g]);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          y[t][s][r] = fmaf(sc[t][s][r], rf[t], -mb[t]);
          top_y = fmaxf(top_y, y[t][s][r]);
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
        sw[s][r] = x.vp[s][r][0];
#pragma unroll
        for (int g = 1; g < kGroups; ++g) sw[s][r] = pgroup == g ? x.vp[s][r][g] : sw[s][r];
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
    for (int byte = 0; byte < kTiles * BITS / 8; ++byte) {
      uint32_t c[4];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        c[2 * s] = byte_pair(x.v[s][0], x.v[s][1], byte);
        c[2 * s + 1] = byte_pair(x.v[s][2], x.v[s][3], byte);
      }
      if constexpr (BITS == 4) {
        auto low = [&](int i) { return centred<4, 0>(c[i] & 0x000f000fu); };
        auto high = [&](int i) { return centred<4, 4>(c[i] & 0x00f000f0u); };
        const f16x8 even = operand(low(0), low(1), low(2), low(3));
        const f16x8 odd = operand(high(0), high(1), high(2), high(3));
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          o[t][2 * byte] = mfma(even, pv[t][2 * byte * 16 / G], o[t][2 * byte]);
          o[t][2 * byte + 1] = mfma(odd, pv[t][2 * byte * 16 / G], o[t][2 * byte + 1]);
        }
      } else {
        auto mid = [&](int i) { return centred<8, 0>(c[i]); };
        const f16x8 a = operand(mid(0), mid(1), mid(2), mid(3));
#pragma unroll
        for (int t = 0; t < NT; ++t) o[t][byte] = mfma(a, pv[t][byte * 16 / G], o[t][byte]);
      }
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

// Combine the four waves of a block that took turns over the keys of the same
// rows: the first wave ends with the sums.
template <int D, int NT, typename W>
__device__ __forceinline__ void join_waves(W& w, float (&l)[NT], int wave, float* lds) {
  constexpr int kRows = NT * 16, kStride = D + 4;
  const int n = threadIdx.x % 16, quad = threadIdx.x / 16 % 4;
  float* ml = lds;                            // [4][kRows][2]
  float* part = lds + kWaves * kRows * 2;     // [2][kRows][kStride]
#pragma unroll
  for (int t = 0; t < NT; ++t)
    if (quad == 0) {
      ml[(wave * kRows + t * 16 + n) * 2] = w.mb[t];
      ml[(wave * kRows + t * 16 + n) * 2 + 1] = l[t];
    }
  __syncthreads();
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    float mm[kWaves], top = kLowest, sum = 0.0f;
#pragma unroll
    for (int v = 0; v < kWaves; ++v) {
      mm[v] = ml[(v * kRows + t * 16 + n) * 2];
      top = fmaxf(top, mm[v]);
    }
#pragma unroll
    for (int v = 0; v < kWaves; ++v)
      sum = fmaf(ml[(v * kRows + t * 16 + n) * 2 + 1], __builtin_amdgcn_exp2f(mm[v] - top), sum);
    const float f = __builtin_amdgcn_exp2f(w.mb[t] - top);
#pragma unroll
    for (int i = 0; i < W::kTiles; ++i) w.o[t][i] *= f;
    w.mb[t] = top;
    l[t] = sum;
  }
#pragma unroll
  for (int half = 2; half >= 1; half /= 2) {
    if (wave >= half && wave < 2 * half) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < W::kTiles; ++i)
          *reinterpret_cast<f32x4*>(part + ((wave - half) * kRows + t * 16 + n) * kStride + i * 16 + quad * 4) = w.o[t][i];
    }
    __syncthreads();
    if (wave < half) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < W::kTiles; ++i)
          w.o[t][i] += *reinterpret_cast<const f32x4*>(part + (wave * kRows + t * 16 + n) * kStride + i * 16 + quad * 4);
    }
    __syncthreads();
  }
}

template <int D, int NT>
constexpr int join_floats() {
  return kWaves * NT * 16 * 2 + 2 * NT * 16 * (D + 4);
}

// grid.x: K/V head fastest, then split, then block of rows (the last rows
// first: under a causal mask they have the most keys); grid.y: sequence.
template <int BITS, int D, int G, int NT, int WR>
__global__ __launch_bounds__(kWaves * 64) void k_kv_attention(KvAttnArgs a) {
  using W = Wave<BITS, D, G, NT>;
  constexpr int kBlockRows = NT * 16 * WR;
  __shared__ float lds[WR == 1 ? join_floats<D, NT>() : 1];
  const int b = blockIdx.y;
  const int hk = blockIdx.x % a.c.kv_heads;
  const int rest = blockIdx.x / a.c.kv_heads;
  const int split = rest % a.plan.splits;
  const int rb = a.plan.row_blocks - 1 - rest / a.plan.splits;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const Seq sq = sequence(a, b);
  const int rows = sq.computed * a.heads_per_kv;
  const int row0 = rb * kBlockRows;
  if (row0 >= rows) return;
  const int row1 = min(row0 + kBlockRows, rows) - 1;
  const Span span = key_span(a, sq.len, sq.n, row0 / a.heads_per_kv, row1 / a.heads_per_kv);
  const int active = (span.tiles + a.plan.split_tiles - 1) / a.plan.split_tiles;
  if (split > 0 && split >= active) return;
  const int base = row0 + (WR == 1 ? 0 : wave * NT * 16);
  if (WR != 1 && base >= rows) return;
  const int last = min(base + NT * 16, rows) - 1;
  // bounds over the wave's rows: a tile inside all of them needs no mask
  const int p0 = sq.len - sq.n + base / a.heads_per_kv, p1 = sq.len - sq.n + last / a.heads_per_kv;
  const int hi_min = a.causal ? p0 : sq.len - 1, hi_max = a.causal ? p1 : sq.len - 1;
  const int lo_max = a.window > 0 ? p1 - a.window + 1 : 0, lo_min = a.window > 0 ? p0 - a.window + 1 : 0;
  const int32_t* table = a.b.page_table + (int64_t)b * a.b.table_stride;

  constexpr int kStep = WR == 1 ? kWaves : 1;
  int t = split * a.plan.split_tiles + (WR == 1 ? wave : 0);
  const int t_end = min((split + 1) * a.plan.split_tiles, span.tiles);
  Tile<BITS, D, G> x, y;
  Pages next;
  // Two buffers, one in flight while the other is worked on.  A load past the
  // last tile repeats it; nothing uses the copy.
  auto fetch = [&](Tile<BITS, D, G>& into, int at) {
    load_tile(into, a.c, next, hk, span.token(min(at, t_end - 1)));
    next = tile_pages(a.c, table, sq.len, span.token(min(at + kStep, t_end - 1)));
  };
  W w;
  auto work = [&](Tile<BITS, D, G>& from, int at) {
    const int tb = span.token(at);
    if (!(tb <= hi_max && (tb + kTile > lo_min || tb < a.sinks))) return;
    const bool whole = tb + kTile - 1 <= hi_min && tb + kTile <= sq.len && from.ok == 3u &&
                       (tb >= lo_max || tb + kTile <= a.sinks);
    w.step(from, tb, !whole, sq.len, a.sinks);
  };
  if (t < t_end) {
    next = tile_pages(a.c, table, sq.len, span.token(t));
    fetch(x, t);
    w.begin(a, sq, hk, base, rows);
    for (;;) {
      fetch(y, t + kStep);
      work(x, t);
      if ((t += kStep) >= t_end) break;
      fetch(x, t + kStep);
      work(y, t);
      if ((t += kStep) >= t_end) break;
    }
  } else {
    w.begin(a, sq, hk, base, rows);
  }
  float l[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) l[i] = w.finish(i);
  if constexpr (WR == 1) {
    join_waves<D, NT>(w, l, wave, lds);
    if (wave != 0) return;
  }
  const int n = threadIdx.x % 16, quad = threadIdx.x / 16 % 4;
#pragma unroll
  for (int t2 = 0; t2 < NT; ++t2) {
    const int row = base + t2 * 16 + n;
    if (row >= rows) continue;
    if (active <= 1) {
      const int i = row / a.heads_per_kv, h = hk * a.heads_per_kv + row - i * a.heads_per_kv;
      const float inv = l[t2] == 0.0f ? 0.0f : 1.0f / l[t2];   // a row that sees nothing becomes 0
      const int64_t e = (int64_t)(sq.first + i) * a.out.row_stride + (int64_t)h * a.out.head_stride + quad * 4;
#pragma unroll
      for (int i2 = 0; i2 < W::kTiles; ++i2) store_out4(a.out, e + i2 * 16, w.o[t2][i2] * inv);
    } else {
      const int64_t at = part_index(a, b, hk, a.plan.row_blocks * kBlockRows, row, split);
      if (quad == 0) {
        a.part_ml[at * 2] = w.mb[t2];
        a.part_ml[at * 2 + 1] = l[t2];
      }
#pragma unroll
      for (int i2 = 0; i2 < W::kTiles; ++i2)
        *reinterpret_cast<f32x4*>(a.part_o + at * D + i2 * 16 + quad * 4) = w.o[t2][i2];
    }
  }
}

}  // namespace kv

namespace {

template <int BITS, int D, int G, int NT, int WR>
hipError_t launch_attention(const KvAttnArgs& a, hipStream_t st) {
  const unsigned blocks = (unsigned)((int64_t)a.c.kv_heads * a.plan.row_blocks * a.plan.splits);
  return kv_launch(kv::k_kv_attention<BITS, D, G, NT, WR>, dim3(blocks, a.b.seqs), dim3(kv::kWaves * 64), st, a);
}

template <int BITS, int D, int G>
hipError_t with_plan(const KvAttnArgs& a, hipStream_t st) {
  const KvPlan& p = a.plan;
  if (p.row_waves == 1) {
    if (p.row_tiles == 1) return launch_attention<BITS, D, G, 1, 1>(a, st);
    if (p.row_tiles == 2) return launch_attention<BITS, D, G, 2, 1>(a, st);
    if constexpr (D <= 128) return launch_attention<BITS, D, G, 4, 1>(a, st);
  } else {
    if (p.row_tiles == 2) return launch_attention<BITS, D, G, 2, 4>(a, st);
    if constexpr (D <= 128) return launch_attention<BITS, D, G, 4, 4>(a, st);
  }
  return hipErrorInvalidValue;   // the plan gives no other form
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
