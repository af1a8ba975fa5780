/*
 * w4a16_step.h -- what a serving step of libw4a16.so (gfx950) runs beside the
 * products (w4a16.h) and the paged 8-bit cache (w4a16_kv.h):
 *
 *   w4a16_qk_norm_rope         per layer, between the q/k/v products and w4a16_kv_append:
 *                              norms of queries and keys for each head, positions rotated in
 *   w4a16_kv_attention_shared  per layer: attention for a batch whose requests begin with the
 *                              same cache entries, read once for all of them
 *   w4a16_sample               once a step: tokens drawn from the LM head's logits
 *
 * Conventions: those of w4a16.h -- device pointers (host ones are named as such), `stream` a
 * hipStream_t as void*, nothing allocated, no state, no synchronization, argument
 * errors before anything is enqueued, deterministic, re-entrant.  Lengths,
 * positions and sampling parameters are read on the device, so the calls can be
 * captured in a graph and replayed as these change.  Sizes 0 succeed without work.
 */
#ifndef W4A16_STEP_H
#define W4A16_STEP_H

#include "w4a16_kv.h"

#ifdef __cplusplus
extern "C" {
#endif

#define W4A16_ROPE_MAX_AXES 4
#define W4A16_ROPE_NORM 1            /* flags of w4a16_qk_norm_rope */
#define W4A16_ROPE_INTERLEAVED 2
#define W4A16_SAMPLE_MAX_ROWS 65536
#define W4A16_SAMPLE_MAX_N (1 << 20)

/*
 * Norm and rotation of a step's queries q [T][HQ][D] and keys k [T][H][D] (bf16,
 * token rows q_stride and k_stride elements apart) into q_out and k_out (bf16,
 * rows q_out_stride and k_out_stride apart):
 *   y = x / sqrt(mean(x^2) + eps) * (weight + weight_offset)     over a head's D elements
 * with W4A16_ROPE_NORM (without it y = x; a NULL weight is a factor of 1), then pair i
 * of the first `rot` elements,
 *   (y[i], y[i + rot / 2])  or with W4A16_ROPE_INTERLEAVED  (y[2i], y[2i + 1]),
 * turned by the angle p * inv_freq[i]: (a cos - b sin, a sin + b cos).  The other
 * elements stay y.  p is positions[t], or with several axes positions[axis][t] of the
 * axis whose section pair i lies in (sections: a HOST array of `axes` pair counts that
 * sum to rot / 2, in order; NULL with one axis).
 *   q_weight, k_weight  bf16 [D];  inv_freq  fp32 [rot / 2];  positions  int32 [axes][T]
 * Squares are summed, factors applied and pairs turned in fp32 (subnormal means and sums
 * count; a head whose squares' sum is beyond fp32 becomes 0); an angle is reduced to one
 * turn in fp64, off by 2^-22 of a turn at most for every int32 position where frequencies
 * are not above 1 (by 2^-25 for positions below 2^20); one rounding to bf16 at the end.
 * H 0 (a layer that reads another's keys) and HQ 0 are allowed, as is rot 0 (no rotation;
 * inv_freq and positions may be NULL).
 * q_out may be q and k_out may be k (with the same stride); otherwise outputs do not
 * overlap inputs.
 * D 64, 128 or 256; rot a multiple of 8, at most D; T <= 2^20; HQ, H <= 2^16.
 * Alignment: q, k, outputs, weights and inv_freq 16 bytes, positions 4, strides multiples of 8 elements.
 */
w4a16_status_t w4a16_qk_norm_rope(const uint16_t *q, int64_t q_stride, const uint16_t *k, int64_t k_stride,
                                  const uint16_t *q_weight, const uint16_t *k_weight, float weight_offset,
                                  const float *inv_freq, const int32_t *positions, const int *sections, int axes,
                                  uint16_t *q_out, int64_t q_out_stride, uint16_t *k_out, int64_t k_out_stride,
                                  float eps, int flags, int tokens, int q_heads, int k_heads, int dim, int rot,
                                  void *stream);

/*
 * Bytes of workspace w4a16_kv_attention_shared needs (0 for invalid arguments): D + 5
 * floats for each part of the shared entries, or chunk of a request's own, and row of `out`.
 */
size_t w4a16_kv_attention_shared_workspace_bytes(int tokens, int requests, int max_new, int max_shared, int max_own,
                                                 int q_heads, const w4a16_kv_cache_t *cache);

/*
 * w4a16_kv_attention (without a window) for decode and verify steps of requests that begin
 * with the same entries: with s = min(max(shared_len[0], 0), max_shared), entry j of every
 * request lies in page
 *   block_table[0][j / P] for j < s,   block_table[r][j / P] from there on,
 * so the shared entries are read once for all requests (those columns of the other rows are
 * not looked at).  s need not end a page.  Partial results are joined for that, which takes
 * longer where shared entries are few: w4a16_kv_attention is faster behind some hundreds of
 * them, by up to a factor of two; from 2000 of them on, 4000 in batches of some 32 requests with
 * heads of 256, this call is as fast or faster, by up to a factor of the requests.
 * Rows, positions and masks are those of w4a16_kv_attention: the row at position pos attends
 * entries 0 .. pos (also where pos < s).
 * max_new bounds the requests' new tokens, max_own their entries from s on (entries from
 * s + max_own on are unread); rows past max_new stay unwritten.
 * max_new * HQ / H must not exceed 64: prompts' many rows read each entry once for many of
 * them in w4a16_kv_attention already (W4A16_ERR_UNSUPPORTED).
 * The arithmetic is w4a16_kv_attention's; the order of sums depends on the call's sizes
 * (tokens, requests, max_*) and s, never on chance.  max_shared, max_own <= 2^28; a call whose
 * chunks of own entries make more than 2^22 workgroups is refused (W4A16_ERR_SHAPE); the
 * other limits and the alignment are w4a16_kv_attention's.
 */
w4a16_status_t w4a16_kv_attention_shared(const uint16_t *q, int64_t q_stride, const w4a16_kv_cache_t *cache,
                                         const int32_t *block_table, int width, const int32_t *seq_lens,
                                         const int32_t *token_start, const int32_t *shared_len, uint16_t *out,
                                         float scale, int tokens, int requests, int max_new, int max_shared,
                                         int max_own, int q_heads, void *workspace, size_t workspace_bytes,
                                         void *stream);

/* Bytes of workspace w4a16_sample needs (0 for invalid arguments): 18.5 KB for each 8192 logits of a row, 152 MB at most
 * (more rows take turns). */
size_t w4a16_sample_workspace_bytes(int M, int N);

/*
 * Draws a token from each row of logits [M][N] (bf16 or fp32 per in_dtype, a w4a16_out_t;
 * rows `stride` elements apart).  With v the row's largest logit and
 *   w[i] = exp((logits[i] - v) / temperature)
 * in 64 bits, and tokens in the order of falling logits (equal ones: lowest index first), a
 * token is kept if
 *   fewer than top_k tokens come before it (top_k <= 0: no limit), and
 *   the weights before it sum to less than top_p times the sum of what top_k keeps
 *   (top_p not below 1: no limit), and
 *   w >= min_p (min_p not above 0: no limit);
 * the first token is always kept.  The drawn one is the first in index order whose
 * running sum of kept weights exceeds u times their sum (the last kept one if none does).
 *   tokens  int32 [M]
 *   share   fp32 [M], or NULL: the drawn token's weight divided by the sum of kept weights
 *   uniforms fp32 [M], in [0, 1); NULL only if temperature is 0 everywhere, which the call
 *           cannot see: NULL uniforms draw the largest logit
 *   temperature, top_p, min_p  fp32 [M], top_k int32 [M]; NULL: 1, 1, 0 and 0 for all rows
 * A temperature that is not above 0 draws the largest logit (lowest index first) with share
 * 1; one above FLT_MAX counts as FLT_MAX.  Logits of -infinity have weight 0 and are never
 * drawn; a row of nothing else gives token -1 and share 0.  With a logit of +infinity only
 * those of +infinity have weight.  A row with a NaN gives its first NaN and share NaN.
 * Sums of weights are of integers, or in a fixed order: the same call gives the same tokens.
 * A weight counts in them to 2^-49 of the row's largest, or to 2^-62 N where that is more
 * (tokens of less may be passed over, also as "the last kept one").  In rows with top_p, min_p or
 * a top_k above 512 the kept weights far in front of a limit, and the sum that top_p is a share
 * of, count to 2^-37 of the largest among 8192 neighbours: sums are off by N 2^-37 of the
 * largest weight at most (2^-17 for 2^20 tokens), and so are top_p's limit, the place that u
 * gives, and share.
 * workspace: w4a16_sample_workspace_bytes(M, N) bytes, not initialised.
 * M <= W4A16_SAMPLE_MAX_ROWS, N <= W4A16_SAMPLE_MAX_N.  N 0: tokens -1, shares 0.
 * Alignment: logits by their type (rows need no more), fp32 and int32 arrays 4, workspace 16.
 */
w4a16_status_t w4a16_sample(const void *logits, int in_dtype, int64_t stride, const float *uniforms,
                            const float *temperature, const int32_t *top_k, const float *top_p, const float *min_p,
                            int32_t *tokens, float *share, void *workspace, size_t workspace_bytes, int M, int N,
                            void *stream);

#ifdef __cplusplus
}
#endif

#endif /* W4A16_STEP_H */
