/*
 * cbs_step.h -- C ABI of what a served transformer block's step does between its
 * linear layers, its paged cache and its attention (cbs_block8.h), on MI355X
 * (gfx950): the residual's addition with the root-mean-square norm, rotary
 * positions, and the pages of the cache by the sequences' lengths.
 *
 * The conventions of conv_bn_silu.h and cbs_block8.h hold: device pointers owned
 * by the caller, nothing kept after the call, work enqueued on `stream` without
 * waiting, every argument validated on the host before any HIP call, a status
 * code returned, nothing thrown.  Handles come from conv_bn_silu_create.
 */
#ifndef CBS_STEP_H
#define CBS_STEP_H

#include <stdint.h>

#include "cbs_block8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* h = x + residual in fp32, rounded to residual_dtype and stored in sum (h = x where residual is
 * NULL); y = h * weight / sqrt(mean over the row of h^2 + eps).
 *   x: [M][K] of dtype (F32, BF16 or F16), row m at x + m * x_stride elements
 *      (x_stride >= K); residual: the same with residual_stride, or NULL; residual_dtype
 *      is dtype or F32 (and ignored where residual is NULL).
 *   weight: contiguous [K] of weight_dtype, which is dtype or F32, or NULL for ones.
 *   eps: 2^-126 or more, finite.
 *   sum: [M][K] of residual_dtype, rows sum_stride apart (>= K); it may be residual itself
 *      (the same pointer and stride).  NULL where residual is NULL.
 *   y: contiguous [M][K] of dtype where y_dtype is dtype; where y_dtype is I8, rows in 8
 *      bits (cbs_rows8_bytes(M, K) bytes, aligned to 16): codes of y before any rounding to dtype.
 * Squares are summed in 64 bits; no finite row overflows or underflows on the way.  A row that holds an
 * infinity gets NaN there and zeros elsewhere, one that holds a NaN gets NaN all over.
 * M = 0 is a no-op.  1 <= K <= 131072 and M <= 2^24, else CBS_ERR_INVALID_ARG (sizes
 * below 1) or CBS_ERR_UNSUPPORTED.  Outputs must not overlap inputs (but sum and residual as
 * said) or each other.  Any alignment to the element size is served. */
int cbs_add_rms_norm(conv_bn_silu_t handle, const void *x, int64_t x_stride, const void *residual,
                     int64_t residual_stride, int residual_dtype, const void *weight, int weight_dtype, float eps,
                     void *sum, int64_t sum_stride, void *y, int y_dtype, int64_t M, int64_t K, int dtype,
                     void *stream);

/* How positions turn a head.  Pair i of the first 2 * pairs dims, (i, i + pairs), or
 * (2i, 2i + 1) where interleaved, becomes
 *   magnitude * (a cos t - b sin t, b cos t + a sin t),   t = position * frequencies[i];
 * the dims past 2 * pairs stay as they are.  t and its reduction are in 64 bits (t is right to
 * 2^-51 of itself), the rest in fp32.
 *   frequencies: fp64 [pairs], radians per position; pairs >= 1. */
typedef struct cbs_rotary {
    const double *frequencies;
    int32_t pairs, interleaved;
    float magnitude;
} cbs_rotary;

/* out = x turned.  x, out: [tokens][heads][dim] of dtype (F32, BF16 or F16), token and head
 * strides in elements (at least dim), dim contiguous; positions: int32 [tokens], of any sign.
 * out may be x itself (the same pointer and strides), else it must not overlap x; its own rows
 * must not overlap.  2 * pairs <= dim <= 512, heads <= 65536, tokens * heads < 2^31. */
int cbs_rotary_apply(conv_bn_silu_t handle, const cbs_rotary *rotary, const void *x, int64_t token_stride,
                     int64_t head_stride, const int32_t *positions, int64_t tokens, int heads, int dim, int dtype,
                     void *out, int64_t out_token_stride, int64_t out_head_stride, void *stream);

/* Queries turned into q_out, keys turned and written into the cache with the values, as
 * cbs_cache_write would write them (rows to 8 bits where it is I8, of the turned key before any
 * rounding to dtype; else converted to its type).
 *   q: [tokens][heads][dim], k, v: [tokens][cache heads][dim] of dtype, dim the cache's; strides as
 *   above.  heads may be 0 (then q and q_out are ignored).  slots as for cbs_cache_write: a token
 *   whose slot lies outside the cache is not written (its queries are turned all the same), and no
 *   two tokens may name one slot.  q_out may be q itself; it may lie between other tensors' rows, as
 *   parts of one wider tensor do, but not on them.
 * 2 * pairs <= dim; heads <= 65536, tokens * (heads + 2 * cache heads) < 2^31. */
int cbs_rotary_cache_write(conv_bn_silu_t handle, const cbs_rotary *rotary, const cbs_paged_cache *cache, const void *q,
                           int64_t q_token_stride, int64_t q_head_stride, const void *k, int64_t k_token_stride,
                           int64_t k_head_stride, const void *v, int64_t v_token_stride, int64_t v_head_stride,
                           const int32_t *positions, const int32_t *slots, int64_t tokens, int heads, int dtype,
                           void *q_out, int64_t out_token_stride, int64_t out_head_stride, void *stream);

/* Pages that no sequence has: free[0 .. counts[0]) is a stack of them, free[pages]; counts: int32 [3],
 * how many there are and, of the last cbs_grow_pages, how many it lacked and how many sequences it left.
 * Both on the device.  A page is free or in one row of the table.  Calls on one pool follow
 * each other: two at once leave it undefined (no access goes out of the tensors). */
typedef struct cbs_page_pool {
    int32_t *free, *counts;
    int64_t pages;
    int32_t page_size;
} cbs_page_pool;

/* Room for more[b] new tokens of each sequence, and where everything lies:
 *   table: int32, row b at table + b * table_stride, table_width entries, the pages of sequence b in
 *      order (entries past its pages hold anything); lens: int32 [batch], its tokens, to which the
 *      new ones are added; more: int32 [batch].
 *   starts: int32 [batch + 1], where each sequence's new tokens begin among the batch's `tokens`;
 *   slots, positions: int32 [tokens], the new tokens' slots (page * page_size + offset) and positions.
 * Negative entries of lens and more count as 0.  Sequences grow in order, each by pages from the top of
 * the stack, as long as there are enough: the first that lacks some, and all after it, are left as
 * they are, as is (alone) one that would pass its row of the table or whose tokens pass `tokens`.
 * Their tokens, and those behind the last sequence's, get the slot -1 and the position 0; where a page
 * of the table or the stack lies outside the pool, the slot is -1.  The tokens of a sequence that is left lie between its
 * starts all the same, and cbs_paged_attention, which goes by lens and knows no slots, takes them for its
 * last old tokens: what it gives for a row whose slot is -1 stands for no token and is not to be used (the slots
 * say on the device which rows those are; the other rows, and what the cache holds, are as they should be, and the
 * tokens can be brought again when there is room).  counts[0] then holds the pages that are
 * left, counts[1] how many more all sequences that fit would have taken, counts[2] how many sequences with new tokens were
 * left.  starts end at `tokens`.
 * batch <= 65536, tokens <= 2^30, pages * page_size < 2^31.  Outputs must not overlap each other or
 * anything else.
 *   workspace: at least cbs_grow_pages_workspace(batch, tokens) bytes, 16-byte aligned; may be NULL for 0. */
int cbs_grow_pages(conv_bn_silu_t handle, const cbs_page_pool *pool, int32_t *table, int64_t table_stride,
                   int64_t table_width, int32_t *lens, const int32_t *more, int64_t batch, int64_t tokens,
                   int32_t *starts, int32_t *slots, int32_t *positions, void *workspace, int64_t workspace_bytes,
                   void *stream);
int64_t cbs_grow_pages_workspace(int64_t batch, int64_t tokens);

/* The sequences keep their first keep[b] tokens (all, where they have no more): lens[b] becomes the smaller
 * of the two (negative ones count as 0), the pages past those tokens go back to the pool and their entries of
 * the table become -1.  An entry that names no page of the pool (a hole that a window has left behind) gives
 * nothing back.  Of all pages given back, in the order of the sequences and of their rows, the first
 * ends on top of the stack: what cbs_grow_pages took and is given back at once lies as it did before.  What
 * does not fit the stack is dropped (then some page was in it twice).
 *   keep: int32 [batch].  Sizes as above; table_width < 2^31.
 *   workspace: at least cbs_release_pages_workspace(batch, table_width) bytes, 16-byte aligned. */
int cbs_release_pages(conv_bn_silu_t handle, const cbs_page_pool *pool, int32_t *table, int64_t table_stride,
                      int64_t table_width, int32_t *lens, const int32_t *keep, int64_t batch, void *workspace,
                      int64_t workspace_bytes, void *stream);
int64_t cbs_release_pages_workspace(int64_t batch, int64_t table_width);

#ifdef __cplusplus
}
#endif

#endif /* CBS_STEP_H */
