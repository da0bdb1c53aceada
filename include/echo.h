/*
 * echo.h -- C ABI of the Echo low-bit all-reduce hot path on one AMD
 * Instinct gfx950 GPU: one rank's share of one all-reduce call.
 *
 * Echo (arXiv 2610.14277) rebuilds a tensor-parallel all-reduce as
 * all-to-all + high-precision sum at the segment owner + all-gather, moves
 * the data as 4-bit (or 8-bit) integers with half-precision group
 * parameters, and feeds the error each call injects back into later calls
 * through two moving averages.  This library holds the per-GPU compute of
 * one call; moving the payloads between GPUs is the caller's job.
 *
 * Pages cited below:
 *   [EA]   "Echo: Error-Compensated 4-Bit Tensor-Parallel Communication for
 *          LLM Training and Inference" -- arXiv abstract.
 *   [JP-W] "テンソル並列の通信を4bitに圧縮する「Echo」" (Japanese explainer),
 *          section "なぜ4bit通信は難しかったのか".
 *   [JP-1] same page, section "Echoの仕組み①" (high-precision sum, low-bit
 *          transport, zero-point-aware asymmetric quantization).
 *   [JP-2] same page, section "Echoの仕組み②" (dual-time-constant feedback
 *          fused into the entry pass).
 *   [JP-F] same page, section "よくある質問" (4-bit integers + half-precision
 *          parameters).
 *
 * Layout (every call):
 *   - A message of n >= 1 elements per rank is split into P contiguous
 *     segments of whole groups: seg_len = echo_segment_len(n, P, group) =
 *     ceil(ceil(n/P) / group) * group, and rank p owns segment p =
 *     [p*seg_len, min((p+1)*seg_len, n)).  When n is a multiple of P*group
 *     every segment holds n/P elements; otherwise the last non-empty segment
 *     ends in a partial group (quantized over its valid elements) and the
 *     segments after it are empty.
 *   - Groups of `group` consecutive elements of a segment (128 by default;
 *     32 and 64 are also accepted) share one scale and one zero point, both
 *     IEEE binary16; params[g] = scale | zero << 16.
 *   - Codes: bits = 4 -> two per byte, the even element in the low nibble
 *     (an odd-length segment leaves its last high nibble 0); bits = 8 -> one
 *     per byte.  Codes and params of a segment are two separate arrays
 *     ("payload", echo_seg), always sized for seg_len elements:
 *     echo_codes_bytes(seg_len, bits) and echo_params_bytes(seg_len, group).
 *   - Dequantized value = fma(code, scale, zero) in fp32.
 *   - Error state: one array per rank of 2n elements of the config's
 *     state type (fp32 or bf16) holding the short memory S and the long
 *     memory L of each element side by side: state[2j] = S_j,
 *     state[2j+1] = L_j.  It is updated in place and persists between
 *     calls (checkpointing it = copying it).
 *
 * Conventions:
 *   - All buffer pointers are device pointers, 16-byte aligned; the caller
 *     owns every buffer.  echo_config and echo_seg arrays are host memory
 *     read during the call only.  The library allocates nothing and keeps
 *     no state between calls; calls on different streams touching disjoint
 *     buffers may run concurrently.
 *   - All calls are asynchronous on `stream` (a hipStream_t; NULL = the
 *     default stream) and never synchronize.
 *   - Payload buffers must not overlap x, the state, the output or each other.
 *   - Every call validates all arguments before touching the GPU and
 *     returns ECHO_OK or a negative error code.  ECHO_ERR_ARG, ECHO_ERR_SHAPE
 *     and ECHO_ERR_ALIGN are returned before anything is launched.  A call
 *     may make more than one launch (the one partial group of a ragged
 *     message runs in a launch of its own, and a segment of more than about
 *     2^33 elements is split over several); ECHO_ERR_HIP can therefore come
 *     after some launches of the call went out, and the state and payloads
 *     it writes may then be partly updated: reset (or restore) the state
 *     before the next call.  No exception crosses this interface.
 */
#ifndef ECHO_H
#define ECHO_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* return codes */
#define ECHO_OK          0
#define ECHO_ERR_ARG    -1   /* null pointer, unsupported or out-of-range parameter */
#define ECHO_ERR_SHAPE  -2   /* n <= 0, or a segment of more than 2^31 groups
                                (every n > 2^48 is one) */
#define ECHO_ERR_ALIGN  -3   /* a buffer pointer is not 16-byte aligned */
#define ECHO_ERR_HIP    -4   /* the HIP runtime reported an error at a launch (earlier
                                launches of the same call may have gone out) */

/* element types */
#define ECHO_IN_BF16     0   /* 16-bit input message: bfloat16 */
#define ECHO_IN_F16      1   /*                       IEEE binary16 */
#define ECHO_OUT_BF16    0   /* all-reduce output: bfloat16 (round to nearest even) */
#define ECHO_OUT_F32     1   /*                    fp32 */
#define ECHO_STATE_F32   0   /* error state S, L: fp32 */
#define ECHO_STATE_BF16  1   /*                   bfloat16 (round to nearest even) */

#define ECHO_MAX_RANKS  16
#define ECHO_GROUP      128  /* default group size; 32 and 64 are also accepted */

typedef struct echo_config {
    int32_t bits;        /* 4 or 8: code width ([JP-F]; 8-bit for early sites) */
    int32_t group;       /* elements per scale/zero pair: 32, 64 or 128 */
    int32_t in_dtype;    /* ECHO_IN_*    */
    int32_t out_dtype;   /* ECHO_OUT_*   */
    int32_t state_dtype; /* ECHO_STATE_* */
    float   eta;         /* feedback gain; finite */
    float   beta_short;  /* decay of the short memory, in [0, 1) */
    float   beta_long;   /* decay of the long memory, in [0, 1) */
    float   mix_long;    /* share of each residual given to the long memory, in [0, 1] */
} echo_config;

/* One segment's payload: codes (seg_len * bits/8 bytes) and params (seg_len/group words). */
typedef struct echo_seg {
    void*     codes;
    uint32_t* params;
} echo_seg;

/*
 * echo_state_reset -- empty both memories: S_j = L_j = +0 for j < n.
 *   state: device array of echo_state_bytes(n, cfg->state_dtype) bytes.
 *   The feedback of [JP-2] carries error into later calls; a chain of calls
 *   starts from an empty state.  Implemented as a fill kernel (no memset
 *   node), so it may be captured in a HIP graph.
 *   Errors: ECHO_ERR_ARG (null cfg/pointer, n <= 0 or n > 2^48, bad state type),
 *   ECHO_ERR_ALIGN, ECHO_ERR_HIP.
 */
int echo_state_reset(const echo_config* cfg, void* state, int64_t n, void* stream);

/*
 * echo_quantize_feedback -- entry pass of rank `rank` ([JP-1], [JP-2]).
 *   For every element j of every segment p != rank:
 *     v = x[j] + eta * (S_j + L_j)                   (fp32, unfused)
 *   each group of v is quantized to `bits` with an fp16 zero point
 *   (the group minimum) and fp16 step ((max - zero) / (2^bits - 1)), codes
 *   round half to even; the payload goes to out[p].  With r = v - dequant:
 *     S_j = beta_short * S_j + (1-beta_short)(1-mix_long) * r
 *     L_j = beta_long  * L_j + (1-beta_long) * mix_long   * r
 *   (each product rounded to fp32, then the sum; the two weights are
 *   computed in double from the float parameters and rounded once).
 *   The owned segment is not read or written (its feedback is applied by
 *   echo_owner_reduce_requant); P = 1 launches nothing.
 *   x: device, n 16-bit elements (in_dtype).  state: device, n (S, L) pairs.
 *   out: host array of P echo_seg; out[rank] is ignored, every other entry
 *   must point at a payload sized for seg_len elements (nothing is written
 *   for an empty segment).
 *   Errors: ECHO_ERR_ARG, ECHO_ERR_SHAPE, ECHO_ERR_ALIGN, ECHO_ERR_HIP.
 */
int echo_quantize_feedback(const echo_config* cfg, int P, int rank, int64_t n,
                           const void* x, void* state,
                           const echo_seg* out, void* stream);

/*
 * echo_owner_reduce_requant -- owner pass of rank `rank` over its segment
 * ([JP-1]: the owner sums in high precision and requantizes; [JP-W]).
 *   For every element j of segment `rank`:
 *     v_own = x[j] + eta * (S_j + L_j)
 *     acc   = sum over p = 0..P-1 in that order of
 *             (p == rank ? v_own : dequant of in[p]'s code for j)    (fp32)
 *   acc is requantized per group into *out (same quantizer as above);
 *   o = the output value of j (bf16-rounded dequant for ECHO_OUT_BF16,
 *   the fp32 dequant for ECHO_OUT_F32); r = acc - o; S_j and L_j are
 *   updated with r as above.  Segments p != rank of x and state are not
 *   read or written.
 *   in: host array of P echo_seg (payloads the other ranks sent for this
 *   segment); in[rank] is ignored.  out: host pointer to one echo_seg.
 *   Errors: ECHO_ERR_ARG, ECHO_ERR_SHAPE, ECHO_ERR_ALIGN, ECHO_ERR_HIP.
 */
int echo_owner_reduce_requant(const echo_config* cfg, int P, int rank, int64_t n,
                              const void* x, void* state,
                              const echo_seg* in, const echo_seg* out, void* stream);

/*
 * echo_dequant_gather -- turn the P owners' requantized payloads into the
 * all-reduce output ([JP-1]: the owner's requantized sum goes to every GPU).
 *   out[p*seg_len + k] = dequant of in[p]'s code k, as out_dtype (bf16
 *   round to nearest even, or fp32), for every p < P and every k below the
 *   element count of segment p (seg_len, fewer in the last non-empty
 *   segment, none after it); nothing past out[n-1] is written.
 *   in: host array of P echo_seg, every entry a valid payload (an empty
 *   segment's payload is not read).  out: device, n elements.
 *   Errors: ECHO_ERR_ARG, ECHO_ERR_SHAPE, ECHO_ERR_ALIGN, ECHO_ERR_HIP.
 */
int echo_dequant_gather(const echo_config* cfg, int P, int64_t n,
                        const echo_seg* in, void* out, void* stream);

/* Sizes (0 for invalid input): the segment length of an n-element message
 * over P ranks, the payload of a segment of seg_len elements, and the error
 * state of an n-element message. */
int64_t echo_segment_len(int64_t n, int P, int group);
size_t echo_codes_bytes(int64_t seg_len, int bits);
size_t echo_params_bytes(int64_t seg_len, int group);
size_t echo_state_bytes(int64_t n, int state_dtype);

/*
 * Quantized K/V cache: keys and values of attention in 4- or 8-bit codes with
 * the quantizer above (group minimum as fp16 zero point, fp16 step, codes round
 * half to even, value = fma(code, step, zero)), written row by row, read back,
 * and read by an attention that works on the codes.
 *
 * The row of one token and K/V head is head_dim elements in groups of `group`.
 * Four arrays hold the cache, codes[num_pages][kv_heads][page_size][head_dim *
 * bits / 8] bytes and params[num_pages][kv_heads][page_size][head_dim / group]
 * words (scale | zero << 16) for keys and for values.  Inside a row the codes
 * are in the order in which the attention kernel's lanes take them: keys as
 * their 8-element runs, run 4 w + i at place i * head_dim / 32 + w; values with
 * element 16 i + m at place m * head_dim / 16 + i; of two 4-bit codes in a byte
 * the earlier place is in the low nibble.  A cache needs no initialization.
 *
 * A call works on the rows of several sequences, packed one after the other:
 * sequence b has the rows row_start[b] .. row_start[b + 1] - 1, and they are its
 * LAST positions: with n = row_start[b + 1] - row_start[b], row i of the n sits
 * at position kv_len[b] - n + i, in slot position % page_size of the page
 * page_table[b * table_stride + position / page_size].  The same description
 * serves writing a step's rows, attending with its queries, and reading rows.
 *
 * The three device arrays cannot be checked by the host.  Whatever they hold,
 * no call leaves the caller's buffers: a row outside every sequence, a position
 * below 0, from max_len on or past the page table, and an entry that names no
 * page are passed over (not written, not read, not attended to); a query row
 * keeps its position there and sees the keys that are left.  Rows behind the
 * last sequence keep their contents.  Two rows of one call in the same slot
 * (a page in two places of the table) leave that slot undefined.
 */
typedef struct echo_kv_cache {
    int32_t   bits;         /* 4 or 8 */
    int32_t   group;        /* 32, 64 or 128, at most head_dim */
    int32_t   head_dim;     /* 64, 128 or 256 */
    int32_t   kv_heads;     /* 1 .. 4096 */
    int32_t   page_size;    /* slots of a page: 16, 32, 64, 128 or 256 */
    int32_t   reserved;     /* not read */
    int64_t   num_pages;    /* 1 .. 2^31 - 1 */
    void*     k_codes;      /* echo_kv_codes_bytes() each */
    void*     v_codes;
    uint32_t* k_params;     /* echo_kv_params_bytes() each */
    uint32_t* v_params;
} echo_kv_cache;

typedef struct echo_kv_batch {
    int32_t seqs;                /* sequences, at most 65535 */
    int32_t rows;                /* rows of the packed arrays, at most 2^30 */
    int32_t max_new;             /* no sequence has more rows (attention: later ones are not computed) */
    int32_t max_len;             /* no kv_len is larger (of a longer sequence, positions from max_len on are passed over) */
    int64_t table_stride;        /* page-table entries per sequence */
    const int32_t* row_start;    /* device, seqs + 1, ascending */
    const int32_t* kv_len;       /* device, seqs: positions in use, this call's rows included */
    const int32_t* page_table;   /* device, seqs * table_stride */
} echo_kv_batch;

/* Packed rows [rows, heads, head_dim], head_dim contiguous, strides in elements.
 * Every row is 16-byte aligned, strides reach 2^40 elements at most; rows that
 * are written share no element. */
#define ECHO_KV_BF16     0
#define ECHO_KV_F16      1
#define ECHO_KV_F32      2
typedef struct echo_kv_rows {
    void*   data;
    int64_t row_stride;
    int64_t head_stride;
    int32_t dtype;          /* ECHO_KV_* */
    int32_t reserved;       /* not read */
} echo_kv_rows;

/*
 * echo_kv_write -- quantize the batch's rows of keys and values into the cache.
 *   k, v: [rows, kv_heads, head_dim], the same type (bf16, fp16 or fp32).
 *   NaN becomes code 0; an infinity the end of the group's range.
 *   Errors: ECHO_ERR_ARG, ECHO_ERR_SHAPE, ECHO_ERR_ALIGN, ECHO_ERR_HIP.
 */
int echo_kv_write(const echo_kv_cache* cache, const echo_kv_batch* batch,
                  const echo_kv_rows* k, const echo_kv_rows* v, void* stream);

/*
 * echo_kv_read -- the batch's rows of keys and values as bf16, fp16 (rounded to
 *   nearest even) or fp32.  Rows the call passes over keep their contents.  k
 *   and v share no element (the same array twice is ECHO_ERR_ARG).
 *   Errors: ECHO_ERR_ARG, ECHO_ERR_SHAPE, ECHO_ERR_ALIGN, ECHO_ERR_HIP.
 */
int echo_kv_read(const echo_kv_cache* cache, const echo_kv_batch* batch,
                 const echo_kv_rows* k, const echo_kv_rows* v, void* stream);

/*
 * echo_kv_attention -- out = softmax(scale * q K^T) V over the cache.
 *   q, out: [rows, q_heads, head_dim], both bf16 or both fp16; query head h
 *   reads K/V head h / (q_heads / kv_heads).  out may be q itself, else they
 *   share no element.  The row at position p sees the keys j < kv_len[b]; with
 *   causal = 1 only j <= p; with window > 0 (causal only) of these only
 *   p - j < window or j < sinks.  Slots that no row sees may hold anything.  A row
 *   that sees nothing becomes 0; one that sees something and has a NaN or infinite
 *   query element, NaN.  scale: finite.
 *   Scores, the softmax and sums are binary32 on the unrounded cached values; a
 *   query element enters within 2^-25 of its row's largest finite one, and
 *   probabilities enter the second product in fp16, relative to the row's maximum.
 *   workspace: echo_kv_workspace_bytes() bytes (may be NULL if that is 0), all 0
 *   when it is first used, and again after a call that failed with
 *   ECHO_ERR_HIP; a completed call leaves it ready for the next, of any sizes
 *   that fit.  Calls that may run at the same time (on other streams, in graphs
 *   replayed side by side) must not share one.
 *   Errors: ECHO_ERR_ARG (also a workspace too small), ECHO_ERR_SHAPE,
 *   ECHO_ERR_ALIGN, ECHO_ERR_HIP.
 */
int echo_kv_attention(const echo_kv_cache* cache, const echo_kv_batch* batch, int q_heads,
                      const echo_kv_rows* q, const echo_kv_rows* out, float scale,
                      int causal, int window, int sinks,
                      void* workspace, size_t workspace_bytes, void* stream);

/* Sizes (0 for invalid input): one codes array and one params array of a cache
 * (its pointers are not read), and the workspace of an attention call (its
 * device arrays are not read; it depends on the sizes only). */
size_t echo_kv_codes_bytes(const echo_kv_cache* cache);
size_t echo_kv_params_bytes(const echo_kv_cache* cache);
size_t echo_kv_workspace_bytes(const echo_kv_cache* cache, const echo_kv_batch* batch, int q_heads,
                               int causal, int window, int sinks);

/* Static description of an error code. */
const char* echo_error_string(int code);

#ifdef __cplusplus
}
#endif

#endif /* ECHO_H */
