/*
 * w4a16_kv.h -- the paged 8-bit key/value cache of libw4a16.so (gfx950): what a
 * decode or prefill step runs between the q/k/v products and the o product of
 * a layer (w4a16.h), in the order of a step
 *
 *   w4a16_kv_plan       once a step: block tables and slot maps from request lengths
 *   w4a16_kv_append     per layer: the new tokens' keys and values into the cache
 *   w4a16_kv_attention  per layer: causal grouped-query attention over the cache
 *   w4a16_kv_dequant    the values of chosen pages (inspection, moving a cache)
 *
 * Letters: R requests, T tokens of this step (all requests', in request order),
 * P tokens a page, H cache heads, HQ query heads (a multiple of H: query head
 * h reads cache head h / (HQ / H)), D the head size.
 *
 * The cache (caller-owned DEVICE memory):
 *   k         8-bit codes [pages][H][P][D]
 *   v         8-bit codes [pages][H][D][P]   (tokens innermost: the attention's
 *                                             second product sums over tokens)
 *   k_scales  bf16 bits   [pages][H]
 *   v_scales  bf16 bits   [pages][H]
 * A key or value is code * scale, code a signed 8-bit integer in -127..127
 * (W4A16_KV_INT8) or an OCP E4M3 number (W4A16_KV_FP8).  For a page and head
 * whose entries' largest magnitude is a, the scale is
 *   INT8: the smallest bf16 number >= a / 127,  FP8: the smallest power of two >= a / 448,
 * at least 2^-100 in both, and a code is the nearest to value / scale, ties to even.
 * (Keys and values are bf16, so value / scale in fp32 never rounds across a tie:
 * the codes are those of exact arithmetic.)
 *
 * Conventions: those of w4a16.h -- device pointers, `stream` a hipStream_t as
 * void*, nothing allocated, no state, no synchronization, argument errors
 * before anything is enqueued, deterministic, re-entrant.  The calls read
 * lengths, tables and slots on the device, so they can be captured in a graph
 * and replayed as these change.
 * Limits: D 64, 128 or 256; P 16, 32, 64, 128 or 256; HQ / H <= 64;
 * pages * P, pages * H and T * HQ < 2^31; H <= 1024; R and T <= 2^20; block
 * tables of at most 2^22 columns; max_len <= 2^29.  Sizes 0 succeed without work.
 * Alignment: q, k, v, out and the codes 16 bytes, strides multiples of 8
 * elements; scales 2; int32 arrays 4; workspace 16; fp32 outputs 16 bytes.
 */
#ifndef W4A16_KV_H
#define W4A16_KV_H

#include "w4a16.h"

#ifdef __cplusplus
extern "C" {
#endif

#define W4A16_KV_MAX_REQUESTS (1 << 20)
#define W4A16_KV_MAX_TOKENS (1 << 20)
#define W4A16_KV_MAX_HEADS 1024
#define W4A16_KV_MAX_GROUP 64
#define W4A16_KV_MAX_WIDTH (1 << 22)
#define W4A16_KV_MAX_DEQUANT ((1 << 24) - 1)    /* pages a w4a16_kv_dequant call */

typedef enum w4a16_kv_type {
    W4A16_KV_INT8 = 0,
    W4A16_KV_FP8 = 1           /* OCP E4M3 (largest 448, no infinities) */
} w4a16_kv_type_t;

typedef struct w4a16_kv_cache {
    void *k;                   /* codes [pages][H][P][D] */
    void *v;                   /* codes [pages][H][D][P] */
    uint16_t *k_scales;        /* bf16 [pages][H] */
    uint16_t *v_scales;        /* bf16 [pages][H] */
    int type;                  /* w4a16_kv_type_t */
    int pages, heads, page, dim;   /* pages, H, P, D */
} w4a16_kv_cache_t;

/*
 * Block tables and slot maps of one step.  Request r holds ctx_lens[r] tokens
 * and brings new_lens[r] (lengths are taken as 0 below 0 and as 2^29 above it;
 * their sums must stay below 2^31).  With held = ceil(ctx / P) and
 * need = ceil((ctx + new) / P) - held, the requests take their pages from
 * free_pages in order:
 *   block_table[r][b]   kept for b < held; then the request's `need` entries
 *                       of free_pages; -1 in the rest of its `width` columns
 *   seq_lens[r]         ctx + new
 *   token_start[R + 1]  exclusive sums of new (token t of request r is row
 *                       token_start[r] + t of the step)
 *   slot_map[T]         page * P + offset of each token's cache entry
 *   pages_used[1]       sum of need
 * Where free_pages has fewer entries than needed (compare pages_used with
 * num_free), or a row fewer columns, the missing entries are -1 and so are
 * the slots in them: w4a16_kv_append skips those.  A page number of 2^31 / P or
 * more is outside every cache, and the slots in it are -1.  Slots past the step's
 * tokens (T may exceed them) are -1; tokens past T have no slot.
 * A caller that drops tokens again (rejected candidates) passes the shorter
 * ctx_lens to the next call and first returns what lies past them to its free
 * pages: entries ceil(kept / P) <= b < ceil(length / P) of the request's row.
 * They are written over, not kept: a page left there would be lost.
 */
w4a16_status_t w4a16_kv_plan(const int32_t *ctx_lens, const int32_t *new_lens, const int32_t *free_pages,
                             int num_free, int32_t *block_table, int width, int32_t *seq_lens,
                             int32_t *token_start, int32_t *slot_map, int32_t *pages_used, int requests,
                             int tokens, int page, void *stream);

/*
 * Quantizes the step's keys and values k, v (bf16 [T][H][D], token rows
 * k_stride and v_stride elements apart: parts of a wider projected row need
 * no copy) into the cache at slot_map's slots.
 * A run is a longest row of tokens with consecutive slots in one page; no two
 * runs of a call may lie in the same page.  A run that begins a page (offset
 * 0) sets the page's scales from its entries; any other keeps the larger of
 * the page's scale and its own, and where the scale grows, the page's codes
 * before the run are encoded again (nearest code of code * old / new).
 * Entries after the run keep their bits.  Slots outside the cache are
 * skipped.  A run with an infinity or NaN sets the page and head's scale to
 * NaN and its codes to 0 (so everything that reads that page sees NaN until
 * it is begun again); a NaN scale stays.
 * A page's scale, and so its codes, depends on how its tokens arrived: on the
 * largest entry of all runs written to it since it was begun, candidates that
 * were rejected later included.  The codes of accepted tokens can therefore
 * differ from those of single-token steps, as they can between a prompt and
 * single tokens, by the rounding of a coarser step.
 */
w4a16_status_t w4a16_kv_append(const uint16_t *k, int64_t k_stride, const uint16_t *v, int64_t v_stride,
                               const int32_t *slot_map, const w4a16_kv_cache_t *cache, int tokens,
                               void *stream);

/*
 * Bytes of workspace w4a16_kv_attention needs (0 is possible, and the answer
 * for invalid arguments): partial results of D + 5 floats for each of up to 128 chunks
 * of max_len entries and each of min(T, R * min(max_new, 64 / (HQ / H))) * HQ rows,
 * and, for few prompt tokens behind a long cache, of D + 2 for each part and row.
 */
size_t w4a16_kv_attention_workspace_bytes(int tokens, int requests, int max_new, int max_len, int window,
                                          int q_heads, const w4a16_kv_cache_t *cache);

/*
 * Causal attention of the step's queries over the cache, the step's own
 * entries included (append first):
 *   out[t][h] = sum_j p_j v_j,  p = softmax_j(scale * q[t][h] . k_j)
 * for row t = token_start[r] + i of request r at position
 * pos = seq_lens[r] - n + i (n = token_start[r + 1] - token_start[r]), over
 * the cache entries 0 <= j <= pos and, with window > 0, j > pos - window.
 * Entry j lies in page block_table[r][j / P]; entries whose page is outside
 * the cache, or past the table's `width` columns, are not attended.  A row
 * without entries is 0.  Rows of q and out outside every request are not
 * touched.  The cache needs at least one page.
 *   q    bf16 [T][HQ][D], token rows q_stride elements apart
 *   out  bf16 [T][HQ][D], dense
 * max_new and max_len bound the requests' n and seq_lens (the launch is sized
 * by them; rows past max_new stay unwritten and entries past max_len unread).
 * Softmax statistics and sums in fp32, weights rounded to fp16, keys, values
 * and queries exact.  A weight is held times its page's value scale: beside
 * values beyond about 10^6 the weights of a page of zeros (scale 2^-100) can
 * underflow.  A row whose logits are all -infinity is 0.
 * Requests of min(n, max_new) * HQ / H <= 64 rows take one form, whose rows
 * depend on their own query, position and entries and on max_len alone: over the
 * same cache they are bitwise equal in any batch and for any number of new tokens
 * up to that bound (a verify batch gives the rows of single-token calls; what it
 * appended may differ, see w4a16_kv_append).  Requests of more take another, as
 * does a call of one request with max_new * HQ / H > 64 (the order of whose sums
 * may depend on the call's sizes, never on chance).
 * (T / (64 / (HQ / H)) + R) * H must not exceed 2^22 (the launch's size).
 */
w4a16_status_t w4a16_kv_attention(const uint16_t *q, int64_t q_stride, const w4a16_kv_cache_t *cache,
                                  const int32_t *block_table, int width, const int32_t *seq_lens,
                                  const int32_t *token_start, uint16_t *out, float scale, int window,
                                  int tokens, int requests, int max_new, int max_len, int q_heads,
                                  void *workspace, size_t workspace_bytes, void *stream);

/*
 * Values (code * scale, exact in fp32) of the pages pages[0 .. count):
 * k_out, v_out fp32 [count][H][P][D], both with tokens outermost.  A page
 * number outside the cache gives NaN.  count is at most W4A16_KV_MAX_DEQUANT.
 */
w4a16_status_t w4a16_kv_dequant(const w4a16_kv_cache_t *cache, const int32_t *pages, int count, float *k_out,
                                float *v_out, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* W4A16_KV_H */
