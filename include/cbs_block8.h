/*
 * cbs_block8.h -- C ABI of the 8-bit operators of a served transformer block
 * on MI355X (gfx950): a linear layer in 8-bit integers, a paged key/value
 * cache that quantises what it is given, and attention over such a cache.
 *
 * The conventions of conv_bn_silu.h hold: device pointers owned by the
 * caller, nothing kept after the call, work enqueued on `stream` without
 * waiting, every argument validated on the host before any HIP call, a status
 * code returned, nothing thrown.  Handles come from conv_bn_silu_create.
 *
 * Rows to 8 bits (shared by the linear layer and the cache).  For a row x:
 *   s = max(fp32(max|x| / 127), 2^-126),   code_i = x_i / s rounded to the
 *   nearest integer, ties to even (of the exact quotient).
 * Codes lie in [-127, 127] and stand for code * s.  A row that holds an
 * infinity or a NaN gets the codes 0 and an infinite or NaN scale, so that it
 * reads back as NaN and the layer's outputs of that row are NaN.
 */
#ifndef CBS_BLOCK8_H
#define CBS_BLOCK8_H

#include <stdint.h>

#include "conv_bn_silu.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types beside CBS_DTYPE_F32 and CBS_DTYPE_BF16. */
enum { CBS_DTYPE_F16 = 2, CBS_DTYPE_I8 = 3 };

/* Activations of the linear layer. */
enum { CBS_ACT_NONE = 0, CBS_ACT_SILU = 1 };

/* y[m][n] = act( (sum_k a[m][k] w[n][k]) * sa[m] * w_scale[n] + bias[n] ),
 * a and sa the rows of x in 8 bits; the sum is exact (32-bit integers), the
 * rest fp32, rounded once to dtype.
 *   x: [M][K] of dtype (F32, BF16 or F16), row m at x + m * x_stride elements
 *      (x_stride >= K); y: contiguous [M][N] of dtype.
 *   w: contiguous int8 [N][K] (any code, -128 included); w_scale: fp32 [N];
 *   bias: fp32 [N] or NULL; activation: CBS_ACT_*.
 *   workspace: at least cbs_int8_linear_workspace(M, N, K) bytes, 16-byte
 *      aligned; its content before and after the call does not matter.  It may
 *      be NULL where that size is 0.
 * M = 0 is a no-op.  1 <= K <= 131072 (the sum then fits 32 bits), 1 <= N,
 * and M, N <= 2^24, else CBS_ERR_INVALID_ARG (sizes below 1) or
 * CBS_ERR_UNSUPPORTED.  y and the workspace must not overlap an input or
 * each other.  Any alignment to the element size is served. */
int cbs_int8_linear(conv_bn_silu_t handle, const void *x, int64_t x_stride, const int8_t *w, const float *w_scale,
                    const float *bias, void *y, int64_t M, int64_t N, int64_t K, int dtype, int activation,
                    void *workspace, int64_t workspace_bytes, void *stream);
/* Bytes of workspace of that call; -1 for sizes it refuses. */
int64_t cbs_int8_linear_workspace(int64_t M, int64_t N, int64_t K);

/* Rows in 8 bits, as cbs_add_rms_norm (cbs_step.h) gives them and the layer below takes them, [M][K]: one
 * buffer of cbs_rows8_bytes(M, K) bytes (-1 for sizes that the layer refuses), aligned to 16:
 *   fp32 scales [R], R = M up to a whole 16;
 *   codes in blocks of 64 along K, [ceil(K / 128) * 2][R][64]: code (m, k) at ((k / 64) * R + m) * 64 + k % 64,
 *   zeros from K on.  What belongs to rows past M may hold anything.
 * So the matrix kernels find the fragments of neighbouring rows side by side. */
int64_t cbs_rows8_bytes(int64_t M, int64_t K);

/* cbs_int8_linear of such rows: the same result as from the x that they were made of.  dtype is
 * that of y.  The workspace is smaller: cbs_int8_linear_rows_workspace(M, N, K), often 0. */
int cbs_int8_linear_rows(conv_bn_silu_t handle, const void *rows, const int8_t *w, const float *w_scale,
                         const float *bias, void *y, int64_t M, int64_t N, int64_t K, int dtype, int activation,
                         void *workspace, int64_t workspace_bytes, void *stream);
int64_t cbs_int8_linear_rows_workspace(int64_t M, int64_t N, int64_t K);

/* A paged cache.  k, v: contiguous [pages][heads][page_size][dim] of dtype (I8,
 * F32, BF16 or F16); k_scale, v_scale: contiguous fp32 [pages][heads][page_size]
 * for I8, NULL otherwise.  A token's slot is page * page_size + offset.
 * k and v (and the scales) are aligned to 16 bytes, dim is a multiple of 8 up
 * to 256, and pages * page_size < 2^31. */
typedef struct cbs_paged_cache {
    void *k, *v;
    float *k_scale, *v_scale;
    int64_t pages;
    int32_t heads, page_size, dim, dtype;
} cbs_paged_cache;

/* Write tokens into the cache: rows to 8 bits where it is I8, else converted to
 * its type (round to nearest even).
 *   k, v: [tokens][heads][dim] of dtype (F32, BF16 or F16), token and head
 *      strides in elements, dim contiguous; slots: int32 [tokens].
 * A token whose slot lies outside [0, pages * page_size) is skipped.  No two tokens
 * of a call may name one slot: what such a slot holds afterwards is undefined (codes
 * of one token may stand under the scale of the other); the other slots are written as
 * ever.  k and v must not overlap the cache. tokens * heads is below 2^31, else
 * CBS_ERR_UNSUPPORTED. */
int cbs_cache_write(conv_bn_silu_t handle, const cbs_paged_cache *cache, const void *k, int64_t k_token_stride,
                    int64_t k_head_stride, const void *v, int64_t v_token_stride, int64_t v_head_stride,
                    const int32_t *slots, int64_t tokens, int dtype, void *stream);

/* Read tokens back: k_out, v_out contiguous [tokens][heads][dim] of dtype;
 * code * scale (or the stored value) rounded once.  A slot outside the cache
 * reads as zeros; tokens may name one slot here.  tokens * heads is below 2^31. */
int cbs_cache_read(conv_bn_silu_t handle, const cbs_paged_cache *cache, const int32_t *slots, int64_t tokens,
                   void *k_out, void *v_out, int dtype, void *stream);

/* Causal attention of each sequence's newest tokens over its cache.
 *   q: [tokens][heads][dim] of dtype (BF16 or F16), token and head strides in
 *      elements; the tokens of sequence b are rows starts[b] .. starts[b+1]-1 and are
 *      the last of its lens[b] tokens (their keys and values are in the cache).
 *   cache: I8, or of q's dtype; heads is a multiple of its heads, head h reads
 *      the cache's head h / (heads / cache heads); dim a multiple of 16.
 *   table: int32, row b at table + b * table_stride holds the pages of sequence
 *      b in order, `table_width` entries; starts: int32 [batch + 1],
 *      non-decreasing; lens: int32 [batch].
 *   window: 0, or the number of latest keys (its own included) that a token sees.
 *   scale: of the scores (1/sqrt(dim) is usual).
 *   out: contiguous [tokens][heads][dim] of dtype.
 * Token i of the new tokens of sequence b, of which there are n, sits at position
 * p = lens[b] - n + i and sees the keys j with p - window < j <= p.
 * out = sum_j softmax_j(scale * q . k_j) v_j; a token that sees no key gets zeros.
 * Keys past lens[b], past the table's width or on a page outside [0, pages) are
 * not seen, and what the cache holds there is never used.  Rows of out that
 * belong to no sequence are left as they are.  starts and lens are read on the
 * device, so the call never waits for them.  tokens * heads up to 2^29, batch *
 * cache heads up to 2^20 (batch up to 65536), table_width * page_size * heads /
 * cache heads up to 2^30, else CBS_ERR_UNSUPPORTED.
 *   workspace: at least cbs_paged_attention_workspace(...) bytes, 16-byte
 *      aligned; content before and after does not matter. */
int cbs_paged_attention(conv_bn_silu_t handle, const void *q, int64_t q_token_stride, int64_t q_head_stride,
                        const cbs_paged_cache *cache, const int32_t *table, int64_t table_stride, int64_t table_width,
                        const int32_t *starts, const int32_t *lens, int64_t batch, int64_t tokens, int heads,
                        int window, float scale, void *out, int dtype, void *workspace, int64_t workspace_bytes,
                        void *stream);
/* Bytes of workspace of that call; -1 for sizes it refuses. */
int64_t cbs_paged_attention_workspace(conv_bn_silu_t handle, int64_t batch, int64_t tokens, int heads, int kv_heads,
                                      int dim, int page_size, int64_t table_width);

#ifdef __cplusplus
}
#endif

#endif /* CBS_BLOCK8_H */
