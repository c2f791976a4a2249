// b8_api.cpp -- the C ABI declared in include/cbs_block8.h: host-side
// validation and kernel launch.  As in cbs_api.cpp, every argument is checked
// before the first HIP call and nothing here allocates or touches device memory.
#include <hip/hip_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "b8_launch.h"
#include "cbs_handle.h"

namespace {

struct Span {
    uintptr_t lo, hi;  // [lo, hi)
};
Span span(const void *p, int64_t bytes) { return {(uintptr_t)p, (uintptr_t)p + (uintptr_t)(p ? bytes : 0)}; }
bool disjoint(Span a, std::initializer_list<Span> others) {
    for (const Span &o : others)
        if (a.lo < o.hi && o.lo < a.hi) return false;
    return true;
}

bool value_type(int dtype) { return dtype == CBS_DTYPE_F32 || dtype == CBS_DTYPE_BF16 || dtype == CBS_DTYPE_F16; }
int64_t element(int dtype) { return dtype == CBS_DTYPE_F32 ? 4 : dtype == CBS_DTYPE_I8 ? 1 : 2; }
bool aligned(const void *p, int64_t to) { return (uintptr_t)p % (uintptr_t)to == 0; }

constexpr int64_t kMaxK = 131072;          // 128 * 128 * K < 2^31
constexpr int64_t kMaxRows = 1 << 24;
constexpr int64_t kMaxStride = 1ll << 40;  // keeps 64-bit offsets exact

int check_linear(int64_t M, int64_t N, int64_t K) {
    if (M < 0 || N < 1 || K < 1) return CBS_ERR_INVALID_ARG;
    if (M > kMaxRows || N > kMaxRows || K > kMaxK) return CBS_ERR_UNSUPPORTED;
    return CBS_OK;
}

// The cache's own fields; its bytes and the spans of its tensors.
int check_cache(const cbs_paged_cache *c) {
    if (!c || c->pages < 1 || c->heads < 1 || c->page_size < 1 || c->dim < 1) return CBS_ERR_INVALID_ARG;
    if (!value_type(c->dtype) && c->dtype != CBS_DTYPE_I8) return CBS_ERR_INVALID_ARG;
    if (!c->k || !c->v) return CBS_ERR_INVALID_ARG;
    if (c->dtype == CBS_DTYPE_I8 ? (!c->k_scale || !c->v_scale) : (c->k_scale || c->v_scale)) return CBS_ERR_INVALID_ARG;
    if (c->pages > INT32_MAX || c->pages * c->page_size > INT32_MAX || c->heads > 65536) return CBS_ERR_UNSUPPORTED;
    if (c->dim % 8 != 0 || c->dim > 256) return CBS_ERR_UNSUPPORTED;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 16) || !aligned(c->v_scale, 16))
        return CBS_ERR_UNSUPPORTED;
    return CBS_OK;
}
int64_t cache_rows(const cbs_paged_cache &c) { return c.pages * c.heads * c.page_size; }
int64_t cache_bytes(const cbs_paged_cache &c) { return cache_rows(c) * c.dim * element(c.dtype); }
bool clear_of_cache(Span s, const cbs_paged_cache &c) {
    return disjoint(s, {span(c.k, cache_bytes(c)), span(c.v, cache_bytes(c)), span(c.k_scale, cache_rows(c) * 4),
                        span(c.v_scale, cache_rows(c) * 4)});
}
bool tensors_disjoint(const cbs_paged_cache &c) {
    const Span k = span(c.k, cache_bytes(c)), v = span(c.v, cache_bytes(c));
    const Span ks = span(c.k_scale, cache_rows(c) * 4), vs = span(c.v_scale, cache_rows(c) * 4);
    return disjoint(k, {v, ks, vs}) && disjoint(v, {ks, vs}) && disjoint(ks, {vs});
}

int check_strides(int64_t tokens, int64_t heads, int64_t dim, int64_t token_stride, int64_t head_stride) {
    (void)tokens;
    if (head_stride < dim && heads > 1) return CBS_ERR_INVALID_ARG;
    if (token_stride < dim && tokens > 1) return CBS_ERR_INVALID_ARG;
    if (token_stride < 0 || head_stride < 0) return CBS_ERR_INVALID_ARG;
    if (token_stride > kMaxStride || head_stride > kMaxStride) return CBS_ERR_UNSUPPORTED;
    return CBS_OK;
}
int64_t strided_bytes(int64_t tokens, int64_t heads, int64_t dim, int64_t token_stride, int64_t head_stride, int dtype) {
    return ((tokens - 1) * token_stride + (heads - 1) * head_stride + dim) * element(dtype);
}

int check_attention_sizes(int64_t batch, int64_t tokens, int64_t heads, int64_t kv_heads, int64_t dim,
                          int64_t page_size, int64_t table_width) {
    if (batch < 0 || tokens < 0 || heads < 1 || kv_heads < 1 || dim < 1 || page_size < 1 || table_width < 0)
        return CBS_ERR_INVALID_ARG;
    if (heads % kv_heads != 0) return CBS_ERR_INVALID_ARG;
    if (dim % 16 != 0 || dim > 256 || heads > 65536 || batch > 65536 || page_size > INT32_MAX ||
        table_width > INT32_MAX)
        return CBS_ERR_UNSUPPORTED;
    // rows (token, head of a group) and positions times the group are 32-bit
    // numbers in the kernels, with room for a tile more
    const int64_t group = heads / kv_heads, lim = 1 << 30;
    if (tokens > lim / group || table_width > lim / group / page_size) return CBS_ERR_UNSUPPORTED;
    // and the launches' workgroups fit a grid
    if (tokens > (1 << 29) / heads || batch > (1 << 20) / kv_heads) return CBS_ERR_UNSUPPORTED;
    return CBS_OK;
}

}  // namespace

extern "C" {

int64_t cbs_int8_linear_workspace(int64_t M, int64_t N, int64_t K) {
    return check_linear(M, N, K) == CBS_OK ? cbs::linear_workspace(M, N, K) : -1;
}

int cbs_int8_linear(conv_bn_silu_t h, const void *x, int64_t x_stride, const int8_t *w, const float *w_scale,
                    const float *bias, void *y, int64_t M, int64_t N, int64_t K, int dtype, int activation,
                    void *workspace, int64_t workspace_bytes, void *stream) {
    if (!cbs::handle_live(h)) return CBS_ERR_BAD_HANDLE;
    if (!value_type(dtype) || (activation != CBS_ACT_NONE && activation != CBS_ACT_SILU)) return CBS_ERR_INVALID_ARG;
    int rc = check_linear(M, N, K);
    if (rc != CBS_OK) return rc;
    if (M == 0) return CBS_OK;
    if (!x || !w || !w_scale || !y || x_stride < K) return CBS_ERR_INVALID_ARG;
    if (x_stride > kMaxStride) return CBS_ERR_UNSUPPORTED;
    const int64_t e = element(dtype), need = cbs::linear_workspace(M, N, K);
    if (need > 0 && (!workspace || workspace_bytes < need)) return CBS_ERR_INVALID_ARG;
    const Span sy = span(y, M * N * e), sw = span(workspace, need);
    const Span in[] = {span(x, ((M - 1) * x_stride + K) * e), span(w, N * K), span(w_scale, N * 4), span(bias, N * 4)};
    for (const Span &i : in)
        if (!disjoint(i, {sy, sw})) return CBS_ERR_INVALID_ARG;
    if (!disjoint(sy, {sw})) return CBS_ERR_INVALID_ARG;
    if (!aligned(x, e) || !aligned(y, e) || !aligned(w_scale, 4) || !aligned(bias, 4) || !aligned(workspace, 16))
        return CBS_ERR_UNSUPPORTED;
    rc = cbs::check_device(h);
    if (rc != CBS_OK) return rc;
    (void)hipGetLastError();
    const cbs::LinearArgs a{x, x_stride, w, w_scale, bias, y, (int)M, (int)N, (int)K, dtype, activation, workspace};
    return cbs::record_hip(cbs::launch_int8_linear(a, (hipStream_t)stream));
}

int cbs_cache_write(conv_bn_silu_t h, const cbs_paged_cache *cache, const void *k, int64_t k_token_stride,
                    int64_t k_head_stride, const void *v, int64_t v_token_stride, int64_t v_head_stride,
                    const int32_t *slots, int64_t tokens, int dtype, void *stream) {
    if (!cbs::handle_live(h)) return CBS_ERR_BAD_HANDLE;
    int rc = check_cache(cache);
    if (rc != CBS_OK) return rc;
    if (!value_type(dtype) || tokens < 0) return CBS_ERR_INVALID_ARG;
    if (tokens > INT32_MAX / cache->heads) return CBS_ERR_UNSUPPORTED;
    if (tokens == 0) return CBS_OK;
    if (!k || !v || !slots || !tensors_disjoint(*cache)) return CBS_ERR_INVALID_ARG;
    for (const auto &s : {std::initializer_list<int64_t>{k_token_stride, k_head_stride}, {v_token_stride, v_head_stride}}) {
        rc = check_strides(tokens, cache->heads, cache->dim, s.begin()[0], s.begin()[1]);
        if (rc != CBS_OK) return rc;
    }
    if (!clear_of_cache(span(k, strided_bytes(tokens, cache->heads, cache->dim, k_token_stride, k_head_stride, dtype)),
                        *cache) ||
        !clear_of_cache(span(v, strided_bytes(tokens, cache->heads, cache->dim, v_token_stride, v_head_stride, dtype)),
                        *cache) ||
        !clear_of_cache(span(slots, tokens * 4), *cache))
        return CBS_ERR_INVALID_ARG;
    if (!aligned(k, element(dtype)) || !aligned(v, element(dtype)) || !aligned(slots, 4)) return CBS_ERR_UNSUPPORTED;
    rc = cbs::check_device(h);
    if (rc != CBS_OK) return rc;
    (void)hipGetLastError();
    const cbs::CacheIo a{*cache, k, v, k_token_stride, k_head_stride, v_token_stride, v_head_stride,
                         nullptr, nullptr, slots, tokens, dtype};
    return cbs::record_hip(cbs::launch_cache_write(a, (hipStream_t)stream));
}

int cbs_cache_read(conv_bn_silu_t h, const cbs_paged_cache *cache, const int32_t *slots, int64_t tokens, void *k_out,
                   void *v_out, int dtype, void *stream) {
    if (!cbs::handle_live(h)) return CBS_ERR_BAD_HANDLE;
    int rc = check_cache(cache);
    if (rc != CBS_OK) return rc;
    if (!value_type(dtype) || tokens < 0) return CBS_ERR_INVALID_ARG;
    if (tokens > INT32_MAX / cache->heads) return CBS_ERR_UNSUPPORTED;
    if (tokens == 0) return CBS_OK;
    if (!k_out || !v_out || !slots) return CBS_ERR_INVALID_ARG;
    const int64_t bytes = tokens * cache->heads * cache->dim * element(dtype);
    const Span sk = span(k_out, bytes), sv = span(v_out, bytes), ss = span(slots, tokens * 4);
    if (!clear_of_cache(sk, *cache) || !clear_of_cache(sv, *cache) || !disjoint(sk, {sv, ss}) || !disjoint(sv, {ss}))
        return CBS_ERR_INVALID_ARG;
    if (!aligned(k_out, element(dtype)) || !aligned(v_out, element(dtype)) || !aligned(slots, 4))
        return CBS_ERR_UNSUPPORTED;
    rc = cbs::check_device(h);
    if (rc != CBS_OK) return rc;
    (void)hipGetLastError();
    const cbs::CacheIo a{*cache, nullptr, nullptr, 0, 0, 0, 0, k_out, v_out, slots, tokens, dtype};
    return cbs::record_hip(cbs::launch_cache_read(a, (hipStream_t)stream));
}

int64_t cbs_paged_attention_workspace(conv_bn_silu_t h, int64_t batch, int64_t tokens, int heads, int kv_heads, int dim,
                                      int page_size, int64_t table_width) {
    if (!cbs::handle_live(h)) return -1;
    if (check_attention_sizes(batch, tokens, heads, kv_heads, dim, page_size, table_width) != CBS_OK) return -1;
    return cbs::attention_workspace(h->num_cu, batch, tokens, heads, kv_heads, dim, page_size, table_width);
}

int cbs_paged_attention(conv_bn_silu_t h, const void *q, int64_t q_token_stride, int64_t q_head_stride,
                        const cbs_paged_cache *cache, const int32_t *table, int64_t table_stride, int64_t table_width,
                        const int32_t *starts, const int32_t *lens, int64_t batch, int64_t tokens, int heads,
                        int window, float scale, void *out, int dtype, void *workspace, int64_t workspace_bytes,
                        void *stream) {
    if (!cbs::handle_live(h)) return CBS_ERR_BAD_HANDLE;
    int rc = check_cache(cache);
    if (rc != CBS_OK) return rc;
    if ((dtype != CBS_DTYPE_BF16 && dtype != CBS_DTYPE_F16) || window < 0 || !std::isfinite(scale))
        return CBS_ERR_INVALID_ARG;
    if (cache->dtype != CBS_DTYPE_I8 && cache->dtype != dtype) return CBS_ERR_UNSUPPORTED;
    rc = check_attention_sizes(batch, tokens, heads, cache->heads, cache->dim, cache->page_size, table_width);
    if (rc != CBS_OK) return rc;
    if (batch == 0 || tokens == 0) return CBS_OK;
    if (!q || !starts || !lens || !out || (!table && table_width > 0) || table_stride < table_width)
        return CBS_ERR_INVALID_ARG;
    if (table_stride > kMaxStride) return CBS_ERR_UNSUPPORTED;
    rc = check_strides(tokens, heads, cache->dim, q_token_stride, q_head_stride);
    if (rc != CBS_OK) return rc;
    const int64_t need = cbs::attention_workspace(h->num_cu, batch, tokens, heads, cache->heads, cache->dim,
                                                  cache->page_size, table_width);
    if (need > 0 && (!workspace || workspace_bytes < need)) return CBS_ERR_INVALID_ARG;
    const Span so = span(out, tokens * heads * cache->dim * element(dtype)), sw = span(workspace, need);
    const Span in[] = {span(q, strided_bytes(tokens, heads, cache->dim, q_token_stride, q_head_stride, dtype)),
                       span(table, ((batch - 1) * table_stride + table_width) * 4), span(starts, (batch + 1) * 4),
                       span(lens, batch * 4)};
    for (const Span &i : in)
        if (!disjoint(i, {so, sw})) return CBS_ERR_INVALID_ARG;
    if (!disjoint(so, {sw}) || !clear_of_cache(so, *cache) || !clear_of_cache(sw, *cache)) return CBS_ERR_INVALID_ARG;
    if (!aligned(q, 2) || !aligned(out, 2) || !aligned(table, 4) || !aligned(starts, 4) || !aligned(lens, 4) ||
        !aligned(workspace, 16))
        return CBS_ERR_UNSUPPORTED;
    rc = cbs::check_device(h);
    if (rc != CBS_OK) return rc;
    (void)hipGetLastError();
    const cbs::AttentionArgs a{q, q_token_stride, q_head_stride, *cache, table, table_stride, (int)table_width,
                               starts, lens, (int)batch, (int)tokens, heads, window, scale, out, dtype, workspace};
    return cbs::record_hip(cbs::launch_paged_attention(a, h->num_cu, (hipStream_t)stream));
}

}  // extern "C"
