/* dckv_cache.h -- a paged KV cache around the codec: rotary positions, writing keys and
 * values into pages, reading pages back as the codec's rows, and attention over the pages.
 *
 * The codec stores pre-RoPE rows of a prompt ("How it works": keys are taken before RoPE,
 * and RoPE is reapplied after decoding).  A serving program keeps the same keys, rotated,
 * in a paged cache.  These calls join the two:
 *   blob --dckv_decode--> K, V --dckv_cache_append--> pages --dckv_attention--> outputs
 *   pages --dckv_cache_rows (keys rotated back)--> rows --dckv_encode--> blob
 * The DCKV method has no counterpart to these calls; head counts, head sizes, rotations and
 * page sizes are the caller's (the codec's own are 6 layers, 2 KV heads, 256 dims, half
 * layout, base 1e7, magnitude 1).
 *
 * Conventions.  As dckv.h: device pointers are caller-owned, calls allocate nothing, are
 * asynchronous and ordered on `stream` (a cudaStream_t, NULL = legacy default stream), make
 * `device` current while they run and give the caller's device back, and return DCKV_OK or a
 * host-detected error before any device work.  They may be captured into a CUDA graph: what
 * a graph fixes is every argument and struct, not the contents of device arrays, so lengths,
 * offsets and page tables may change between replays.
 * Structs are host memory, read during the call only.  Strides are in elements; the last
 * dimension of every tensor is contiguous.
 *
 * Status.  *status (device int32) is written only when an error is found on the device
 * (unlike dckv_encode's, which every call overwrites): set it to 0 once, and one word can
 * collect the errors of many calls.  DCKV_ERANGE: a length, offset or page index is outside
 * its bounds; nothing is read or written out of bounds, and the tokens concerned are left out
 * (dckv_attention: of a sequence with a bad length or offset; the slots of a bad page count as
 * zero keys and values).  DCKV_ETIMEOUT as in dckv.h: the call's outputs are undefined. */
#ifndef DCKV_CACHE_H_
#define DCKV_CACHE_H_

#include <stddef.h>
#include <stdint.h>

#include "dckv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- element types ---- */
#define DCKV_BF16 0
#define DCKV_FP16 1
#define DCKV_FP32 2 /* dckv_rope only */

/* ---- rotary positions ---- */
#define DCKV_ROPE_MAX_PAIRS 128
#define DCKV_ROPE_HALF 0        /* pairs (i, i + rotary_dim / 2), the codec's layout       */
#define DCKV_ROPE_INTERLEAVED 1 /* pairs (2 i, 2 i + 1)                                    */
#define DCKV_ROPE_NONE 0        /* f_i = base^(-2 i / rotary_dim)                          */
#define DCKV_ROPE_LINEAR 1      /* f_i / factor                                            */
#define DCKV_ROPE_NTK 2         /* base * factor^(rotary_dim / (rotary_dim - 2))           */
#define DCKV_ROPE_PARTS 3       /* f_i * (w + (1 - w) / factor) with
                                   w = clamp((t - low) / (high - low), 0, 1) and
                                   t = original_len f_i / (2 pi), the turns that pair i makes
                                   within the trained length (the ramp is linear in turns; one
                                   linear in i gives other frequencies: fill freq by hand) */
#define DCKV_ROPE_FORWARD 0     /* a' = m (a cos - b sin),  b' = m (b cos + a sin)         */
#define DCKV_ROPE_GRADIENT 1    /* its transpose: a' = m (a cos + b sin), b' = m (b cos - a sin);
                                   the gradient of x from the gradient of the output       */
#define DCKV_ROPE_INVERSE 2     /* its inverse: the transpose with 1 / m in place of m     */

/* A rotation: angle of pair i at position p = p * freq[i] radians (multiplied and reduced to
 * within a turn in fp64), cos and sin in fp32, times `magnitude` m.  Dims past
 * rotary_dim are not rotated.  Filled by dckv_rope_init, or by the caller. */
typedef struct {
  int32_t rotary_dim; /* even, 2 .. 2 * DCKV_ROPE_MAX_PAIRS                                */
  int32_t layout;     /* DCKV_ROPE_HALF or DCKV_ROPE_INTERLEAVED                           */
  double magnitude;   /* 2^-126 .. 2^126                                                   */
  double freq[DCKV_ROPE_MAX_PAIRS]; /* the first rotary_dim / 2 are used                   */
} dckv_rope_spec;

/* Fills *out (host only).  base > 1; factor > 0 (not used by DCKV_ROPE_NONE); original_len > 0
 * and high > low for DCKV_ROPE_PARTS; DCKV_ROPE_NTK needs rotary_dim > 2. */
int dckv_rope_init(dckv_rope_spec *out, int rotary_dim, int layout, double base, int scaling, double factor,
                   double original_len, double low, double high, double magnitude);

/* Rotates x [n_tokens][n_heads][head_dim] (DCKV_BF16, DCKV_FP16 or DCKV_FP32; fp32
 * arithmetic, one rounding) by positions (any int32) into out, same shape and type.  out may be x
 * itself with x's strides (in place); otherwise the byte ranges that x and out span must not
 * overlap. */
typedef struct {
  const void *x; /* device, aligned to its elements                                        */
  void *out;
  int64_t x_token_stride, x_head_stride, out_token_stride, out_head_stride;
  int64_t n_tokens; /* up to 2^31 - 1                                                      */
  int32_t n_heads;  /* up to 65,535                                                        */
  int32_t head_dim; /* rotary_dim .. 65,536                                                */
  const int32_t *positions; /* device int32 [n_tokens]                                     */
  int32_t dtype;
  int32_t device;
} dckv_rope_args;

int dckv_rope(const dckv_rope_spec *spec, int mode, const dckv_rope_args *args, void *stream);

/* ---- the paged cache ---- */

/* Page pools of keys and values: k[layer][page][row][head][dim] at
 *   k + layer * k_layer_stride + page * k_page_stride + row * k_row_stride + head * k_head_stride
 * (rows or heads outermost within a page, or any other strides), v likewise. */
typedef struct {
  void *k, *v;        /* device, 16-byte aligned                                           */
  int32_t device;
  int32_t dtype;      /* DCKV_BF16 or DCKV_FP16                                            */
  int32_t n_layers, n_kv_heads;
  int32_t head_dim;   /* 64, 128 or 256                                                    */
  int32_t page_size;  /* rows per page, a multiple of 16 up to 65,536                      */
  int64_t n_pages;    /* up to 2^31 - 1                                                    */
  int64_t k_layer_stride, k_page_stride, k_row_stride, k_head_stride; /* multiples of 8    */
  int64_t v_layer_stride, v_page_stride, v_row_stride, v_head_stride;
} dckv_kv_pool;

/* The sequences of a call.  Tokens of all sequences stand one after the other: sequence b
 * has tokens offsets[b] .. offsets[b+1] - 1 of the call's token tensors (n_b of them).  Slot j
 * of a sequence (its j-th cached token) is row j % page_size of page
 * page_table[b * table_stride + j / page_size]; entries past a sequence's last page are never
 * read.  kv_lens[b] counts the slots in use.  Tokens from offsets[batch] on belong to no
 * sequence and their outputs are left as they were. */
typedef struct {
  int32_t batch;      /* 1 .. DCKV_MAX_PROMPTS                                             */
  int32_t max_new;    /* host bound of n_b, 1 .. 2^30 (DCKV_ERANGE where n_b is larger); attention
                         looks at row tiles up to it, so a far larger one costs time        */
  int32_t max_pages;  /* columns of page_table                                             */
  int32_t reserved;   /* 0                                                                 */
  const int32_t *offsets;    /* device [batch + 1], non-decreasing                         */
  const int32_t *kv_lens;    /* device [batch]                                             */
  const int32_t *page_table; /* device [batch][max_pages]                                  */
  int64_t table_stride;
} dckv_cache_batch;

/* Writes n_tokens new keys and values [n_layers][n_tokens][n_kv_heads][head_dim] (the pool's
 * type, strides multiples of 8 elements, 16-byte aligned) into the pages: token t of sequence
 * b goes to slot kv_lens[b] - n_b + t (kv_lens counts the new tokens).  With `rope` keys are
 * rotated (forward) on their way, at position positions[token] or, where positions (device
 * int32 [n_tokens]) is NULL, at their slot; without it they are copied.  With q (device
 * [n_tokens][n_q_heads][head_dim], needs rope), q is rotated at the same position into q_out,
 * which may be q itself with its strides, or must not overlap it.  k, v, q and q_out must not
 * overlap the pools, nor q_out k and v, and two tokens of one call must not share a slot.  With
 * n_b = kv_lens[b] and no rope this takes over what dckv_decode wrote: layer stride
 * n_tokens * 512, token stride 512, head stride 256. */
typedef struct {
  const void *k, *v;
  int64_t k_layer_stride, k_token_stride, k_head_stride;
  int64_t v_layer_stride, v_token_stride, v_head_stride;
  const void *q; /* may be NULL (q_out is then ignored)                                    */
  void *q_out;
  int64_t q_token_stride, q_head_stride, q_out_token_stride, q_out_head_stride;
  int64_t n_tokens;          /* up to 2^31 - 1                                             */
  int32_t n_q_heads;         /* up to 65,535                                               */
  int32_t reserved;          /* 0                                                          */
  const int32_t *positions;  /* may be NULL                                                */
} dckv_append_args;

int dckv_cache_append(const dckv_kv_pool *pool, const dckv_cache_batch *batch, const dckv_rope_spec *rope,
                      const dckv_append_args *args, int32_t *status, void *stream);

/* Reads the first n_b = offsets[b+1] - offsets[b] slots of each sequence (n_b <= kv_lens[b])
 * as rows [n_layers][K, V][n_kv_heads][head_dim], token stride row_stride elements (a multiple
 * of 8; rows 16-byte aligned, the pool's type): with the codec's 6 layers, 2 heads and 256 dims
 * these are dckv_encode's rows.  With `rope` keys are rotated back (inverse; fp32, one rounding)
 * from position positions[token] or, where that is NULL, from their slot.  max_new is not used. */
int dckv_cache_rows(const dckv_kv_pool *pool, const dckv_cache_batch *batch, const dckv_rope_spec *rope, void *rows,
                    int64_t row_stride, int64_t n_tokens, const int32_t *positions, int32_t *status, void *stream);

/* ---- attention ---- */

/* out[t][h] = sum_j softmax_j(scale q[t][h] . k[j][h / g]) v[j][h / g] over the slots j that
 * token t of sequence b sees: all j < kv_lens[b], or with `causal` those with
 * j <= kv_lens[b] - n_b + t (the new tokens are the sequence's last, already appended);
 * g = n_q_heads / n_kv_heads.  A token that sees no slot gets out = 0 and lse = -infinity;
 * one that sees slots and whose query holds NaN gets NaN in both.
 * lse (natural logarithm of sum_j exp(scale q . k)) allows outputs over disjoint sets of slots
 * to be joined.  Slots that a sequence does not use may hold anything; keys and values that
 * are in use must be finite (a value beyond the causal bound of one row may still be
 * multiplied by that row's weight 0).
 * Scores, maxima, sums and outputs are fp32; the weights are rounded to the cache's type before
 * they multiply v (by at most half a step of each weight; in fp16 a weight below 2^-21 of the row's
 * largest by at most 2^-32 of that one), and out is rounded once.
 * One kernel serves a whole call, chosen by max_new times g: single tokens that share a call with a
 * long chunk run on its 256-row tiles, so a caller that has both gains by two calls (up to 1.45
 * times on 63 tokens beside a chunk of 512 at dim 64, 1.05 times at dim 256).
 * For a given device and arguments, the result is the same on every call; a sequence's bits
 * may depend on the other sequences of the call, which decide where its slots are split. */
typedef struct {
  const void *q;   /* device [n_tokens][n_q_heads][head_dim], the pool's type, 16-byte aligned */
  void *out;       /* same shape and type, must not overlap q                              */
  float *lse;      /* device fp32 [n_tokens][n_q_heads], contiguous; may be NULL           */
  int64_t q_token_stride, q_head_stride, out_token_stride, out_head_stride; /* multiples of 8 */
  int64_t n_tokens;   /* up to 2^31 - 1                                                    */
  int32_t n_q_heads;  /* a multiple of n_kv_heads                                          */
  int32_t layer;
  int32_t causal;     /* 0 or 1                                                            */
  float scale;        /* finite, > 0                                                       */
} dckv_attention_args;

/* Workspace bytes for dckv_attention on this pool, batch and head count (0 on bad arguments).
 * It depends on max_new, not on the lengths: up to 3 MB where max_new * g is small (8, or 16
 * below dim 256), else up to 43 MB.  256-byte aligned; its contents need no preparation; calls that may overlap in time
 * (two streams, two graphs) need one each. */
size_t dckv_attention_workspace_bytes(const dckv_kv_pool *pool, const dckv_cache_batch *batch, int n_q_heads);

int dckv_attention(const dckv_kv_pool *pool, const dckv_cache_batch *batch, const dckv_attention_args *args,
                   int32_t *status, void *workspace, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* DCKV_CACHE_H_ */
