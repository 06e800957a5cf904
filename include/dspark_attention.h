/*
 * dspark_attention.h - C ABI of the cache side of a verify cycle on B200 (sm_100a): the rotary
 * embedding and append of each sequence's new tokens, and their attention over its paged cache.
 *
 * The verify forward that makes p_2..p_{K+1} (dspark_verify.h, rows 1..K of the logit block)
 * runs a few new tokens per sequence, the anchor and its drafts, against a long cache; the
 * same two operators serve a plain decode step (one new token) and a chunk of a prompt
 * (thousands). The cycle: append the block's keys and values behind the accepted context
 * (kv_len counts them), attend, verify, then set kv_len to the accepted length: the slots of
 * rejected drafts are written again by the next cycle.
 *
 * Rules that hold for both calls
 * ------------------------------
 *  - Device pointers, a cudaStream_t as `stream`, no allocation, no synchronisation, no host
 *    read of device data: a call can be captured into a CUDA graph. It runs on the CURRENT
 *    device, which must hold the buffers.
 *  - Argument errors return a code and enqueue nothing. What only the device can see (a count,
 *    a length or a page id out of range) is reported per sequence in `status` and never reads
 *    or writes out of range.
 *  - Strides are in elements; the last dimension (head_dim) is contiguous.
 *  - Both kernels are programmatic dependent launches that wait for the kernel before them.
 */
#ifndef DSPARK_ATTENTION_H
#define DSPARK_ATTENTION_H

#include "dspark_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Per-sequence bits of `status` (beside DSPARK_SEQ_BAD_PARAM of dspark_verify.h: a count,
 * start or length out of range; nothing of the sequence is read or written). */
#define DSPARK_SEQ_BAD_PAGE 32 /* a page id outside [0, n_pages) among the pages the call needs */

/* One tensor of head rows: token i of sequence b, head h starts at
 * p + b * seq_stride + i * token_stride + h * head_stride (packed rows: seq_stride unused, i
 * counts from the first token of the call). */
typedef struct {
  void* p;
  int64_t seq_stride, token_stride, head_stride;
} dspark_heads_t;

/* The new tokens of the call's B sequences, in one of two forms.
 *  Block (q_start == NULL): tensors are [B, N, heads, head_dim]; sequence b has n_new[b] new
 *    tokens, 0 <= n_new[b] <= N (n_new == NULL: N everywhere), its first rows.
 *  Packed (q_start != NULL): tensors are [N, heads, head_dim]; sequence b has the rows
 *    q_start[b] .. q_start[b+1] - 1, 0 <= q_start[b] <= q_start[b+1] <= N. n_new must be NULL.
 * Rows that belong to no sequence have no effect and are never written. Starts that are out of
 * range or decrease make their own sequence DSPARK_SEQ_BAD_PARAM and leave the others as they
 * would be without it; rows that two sequences then share hold the result of either. */
typedef struct {
  int B, N;
  const int32_t* n_new;   /* device [B] or NULL */
  const int32_t* q_start; /* device [B+1] or NULL */
} dspark_rows_t;

/* The paged cache of one layer. Token position t of sequence b sits in page
 * page_table[b * ld_table + t / page_size], slot t % page_size; that slot's key of head h is at
 * k + page * k_page_stride + slot * k_token_stride + h * k_head_stride (values likewise), so
 * [pages, slots, heads, head_dim] and [pages, heads, slots, head_dim] are both accepted.
 * kv_len[b] counts the tokens of the sequence, the new ones included: new token i sits at
 * position kv_len[b] - n + i. 0 <= kv_len[b] <= max_pages * page_size <= 2^30. Entries past the
 * last needed page are never read. */
typedef struct {
  void* k;
  void* v;
  int64_t k_page_stride, k_token_stride, k_head_stride;
  int64_t v_page_stride, v_token_stride, v_head_stride;
  int n_pages, page_size, n_heads, head_dim;
  const int32_t* page_table; /* device [B, max_pages] */
  int64_t ld_table;
  int max_pages;
  const int32_t* kv_len; /* device [B] */
} dspark_kv_cache_t;

/* Scalings of the rotary frequencies for contexts beyond the trained one. */
typedef enum {
  DSPARK_ROTARY_PLAIN = 0,  /* theta^(-2i/R)                                              */
  DSPARK_ROTARY_LINEAR = 1, /* every frequency divided by `factor` (position interpolation) */
  DSPARK_ROTARY_NTK = 2,    /* theta raised to theta * factor^(R / (R - 2))                */
  DSPARK_ROTARY_YARN = 3,   /* a ramp between plain and divided frequencies over the number
                               of turns in the trained context, and a magnitude            */
  DSPARK_ROTARY_BANDS = 4   /* low frequencies divided, high ones kept, a smooth band between
                               in the number of turns in the trained context               */
} dspark_rotary_scaling_t;

/* The R/2 rotary frequencies (radians per token) on the HOST, computed in double and rounded
 * once to float, and the factor of the rotated values (1 but for YARN).
 *  R        rotated elements of a head, even, 2..1024.
 *  theta    the base, > 1.
 *  factor   how many times the trained context is exceeded, >= 1 (unused by PLAIN).
 *  trained  the trained context in tokens, >= 1 (YARN and BANDS).
 *  low, high  turns in the trained context that bound the ramp, 0 < low < high (YARN: fast and
 *           slow ends, commonly 1 and 32; BANDS commonly 1 and 4).
 *  YARN: frequency f_i makes r_i = trained f_i / (2 pi) turns; the index at which r turns are
 *   made is d(r) = R log(trained / (2 pi r)) / (2 log theta); g_i = clamp((i - floor d(high)) /
 *   (ceil d(low) - floor d(high)), 0, 1) (bounds clamped to [0, R - 1]); the frequency is
 *   (1 - g_i) f_i + g_i f_i / factor; the magnitude 0.1 ln(factor) + 1.
 *  BANDS: g_i = clamp((r_i - low) / (high - low), 0, 1), the frequency g_i f_i + (1 - g_i)
 *   f_i / factor. */
dspark_status_t dspark_rotary_frequencies(int R, double theta, dspark_rotary_scaling_t scaling,
                                          double factor, double trained, double low, double high,
                                          float* inv_freq, float* magnitude);

/* Rotary embedding of the new tokens, and their append to the cache.
 *  q [.., n_q_heads, head_dim] is rotated into q_out (which may be q itself); k and v
 *  [.., cache.n_heads, head_dim]: the rotated k and v as they are go to the tokens' slots.
 *  The first R elements of each head turn; the others are copied. A pair (x1, x2) at angle
 *  a = position * inv_freq[i] becomes magnitude * (x1 cos a - x2 sin a, x2 cos a + x1 sin a);
 *  the pairs are elements (i, i + R/2), or (2i, 2i + 1) when `interleaved`.
 *  The angle is reduced to a turn in float64, so far positions lose nothing; the rotation is
 *  float32, rounded once to `dtype` (DSPARK_BF16 or DSPARK_F16).
 *  inv_freq  device float [R/2], R even in [0, head_dim], head_dim <= 1024 (R == 0: no rotation,
 *            inv_freq may be NULL).
 *  A sequence needs kv_len[b] >= n (else DSPARK_SEQ_BAD_PARAM). A packed row that two sequences
 *  claim (where starts decrease) is appended for one of them; a sequence that may lack such a
 *  row is DSPARK_SEQ_BAD_PARAM, though its other rows are appended. A token whose page id is out
 *  of range is not appended (DSPARK_SEQ_BAD_PAGE); its query is rotated as usual.
 *  status    device [B] or NULL: 0 or DSPARK_SEQ_* bits.
 *  No workspace. Slots must not be shared by two new tokens (their order is not defined). */
dspark_status_t dspark_rotary_append(dspark_heads_t q, int n_q_heads, dspark_heads_t q_out,
                                     dspark_heads_t k, dspark_heads_t v, dspark_dtype_t dtype,
                                     dspark_kv_cache_t cache, dspark_rows_t rows,
                                     const float* inv_freq, int R, int interleaved,
                                     float magnitude, int32_t* status, void* stream);

/* Attention of the new tokens over the paged cache (their own keys and values appended).
 *  q, out    [.., n_q_heads, head_dim] of `dtype` (DSPARK_BF16 or DSPARK_F16, the cache's type
 *            too); query head h reads cache head h / (n_q_heads / n_heads). out may be q itself.
 *  New token i of sequence b, at position p = kv_len[b] - n + i, sees the positions t < kv_len[b]
 *  with t <= p when `causal`, and t > p - window when window > 0; out = sum_t w_t v_t with
 *  w = softmax over the seen t of scale * q . k_t. A token that sees nothing gives zeros (and
 *  lse -inf). Keys and values that a token does not see do not affect it, whatever they hold;
 *  a non-finite value that it sees makes (at least) that element of its result non-finite.
 *  scale     finite, > 0.
 *  lse       device float [rows, n_q_heads] (block: [B, N, heads], packed: [N, heads]) or NULL:
 *            log of the sum of exp(scale * q . k_t) over the seen t (natural logarithm).
 *  status    device [B] or NULL. A token that sees a position whose page id is out of range
 *            gives NaN (DSPARK_SEQ_BAD_PAGE); the others are not affected. When the kernel gives up
 *            on one of its (bounded) waits every sequence has DSPARK_SEQ_TIMEOUT: rows may be
 *            unwritten or NaN, and dspark_pipeline_timeouts grows.
 *  Limits (else DSPARK_ERR_UNSUPPORTED): head_dim a multiple of 8 in [16, 128]; page_size a
 *  power of two in [8, 1024]; at most 4096 heads and 65535 sequences; pointers and strides
 *  multiples of 16 bytes, the cache's strides below 2^40 bytes.
 *  Numerics: scores and sums in float32 (products on the tensor cores, their sums moved on
 *  before the cut-off there adds up to a quarter or half of the type's half step); the weights
 *  are rounded to `dtype` for the product with v, the statistics are not. A weight is off by a
 *  relative 2^-8 (bf16), or by a relative 2^-11 and 2^-37 of the row's largest weight (f16: with
 *  equal small weights beside one large, noticeable from some 2^26 positions on). out is rounded
 *  once, and finite values give a finite out (bf16: where 2^8 kv_len |v| stays below 2^127, as
 *  the weighted values are summed before the division). A row whose seen scores are all -inf
 *  gives zeros and lse -inf, as one that sees nothing.
 *  workspace  dspark_block_attention_workspace_bytes bytes, 256-byte aligned, no
 *            initialisation; one workspace serves one call at a time. */
size_t dspark_block_attention_workspace_bytes(int N, int n_q_heads, int n_heads, int head_dim);
dspark_status_t dspark_block_attention(dspark_heads_t q, int n_q_heads, dspark_heads_t out,
                                       dspark_dtype_t dtype, dspark_kv_cache_t cache,
                                       dspark_rows_t rows, float scale, int causal, int window,
                                       float* lse, int32_t* status, void* workspace,
                                       size_t workspace_bytes, void* stream);

/* For tests of the timeout path only: dspark_block_attention with each CTA's first copy of keys
 * withheld, so that the waits for it run out (about a second) and the kernel gives up: the call
 * returns DSPARK_OK, its outputs are incomplete, every sequence has DSPARK_SEQ_TIMEOUT and
 * dspark_pipeline_timeouts grows. */
dspark_status_t dspark_block_attention_withheld(dspark_heads_t q, int n_q_heads,
                                                dspark_heads_t out, dspark_dtype_t dtype,
                                                dspark_kv_cache_t cache, dspark_rows_t rows,
                                                float scale, int causal, int window, float* lse,
                                                int32_t* status, void* workspace,
                                                size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DSPARK_ATTENTION_H */
