// st_api.cpp -- the C ABI declared in include/cbs_step.h: host-side validation and kernel
// launch.  As in b8_api.cpp, every argument is checked before the first HIP call and nothing here
// allocates or touches device memory.
#include <hip/hip_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "b8_checks.h"
#include "cbs_handle.h"
#include "st_launch.h"

namespace {

using namespace cbs;

constexpr int64_t kMaxK = 131072, kMaxRows = 1 << 24;  // as the linear layer's
constexpr int kMaxDim = 512, kMaxHeads = 65536;

// A tensor [tokens][heads][dim] as the rotary operators take it.
struct Heads {
    const void *p;
    int64_t token, head;  // strides in elements
    int64_t tokens, heads, dim, e;
    Span all() const { return span(p, ((tokens - 1) * token + (heads - 1) * head + dim) * e); }
    int64_t extent() const { return ((heads - 1) * head + dim) * e; }  // bytes of one token
    bool same(const Heads &o) const {
        return p == o.p && (token == o.token || tokens <= 1) && (head == o.head || heads <= 1);
    }
    // Whether no two rows share memory.
    bool apart() const {
        return tokens <= 1 || heads <= 1 || token >= (heads - 1) * head + dim || head >= (tokens - 1) * token + dim;
    }
    // Whether the two share no memory: they lie apart, or between each other's tokens or heads.
    bool beside(const Heads &o) const {
        if (disjoint(all(), {o.all()})) return true;
        if (e != o.e) return false;
        const bool tokens_alike = tokens > 1 && token == o.token, heads_alike = heads > 1 && head == o.head;
        if (tokens_alike && between(o, token * e, extent(), o.extent())) return true;
        if (heads_alike && between(o, head * e, ((tokens - 1) * token + dim) * e, ((o.tokens - 1) * o.token + o.dim) * e)) return true;
        // every row begins at a multiple of the head stride from the first
        return heads_alike && (tokens <= 1 || (tokens_alike && token % head == 0)) && between(o, head * e, dim * e, o.dim * e);
    }
    // Whether blocks of `mine` and `its` bytes, each repeated with this period, miss each other.
    bool between(const Heads &o, int64_t period, int64_t mine, int64_t its) const {
        int64_t at = (int64_t)((uintptr_t)o.p - (uintptr_t)p) % period;
        if (at < 0) at += period;
        return mine <= at && at + its <= period;
    }
};

int check_rotary(const cbs_rotary *r, int64_t dim) {
    if (!r || !r->frequencies || r->pairs < 1 || !std::isfinite(r->magnitude)) return CBS_ERR_INVALID_ARG;
    if ((int64_t)r->pairs * 2 > dim) return CBS_ERR_INVALID_ARG;
    return aligned(r->frequencies, 8) ? CBS_OK : CBS_ERR_UNSUPPORTED;
}
Span frequencies_of(const cbs_rotary &r) { return span(r.frequencies, (int64_t)r.pairs * 8); }

int check_pool(const cbs_page_pool *p) {
    if (!p || !p->free || !p->counts || p->pages < 1 || p->page_size < 1) return CBS_ERR_INVALID_ARG;
    if (p->pages > INT32_MAX || p->pages * p->page_size > INT32_MAX) return CBS_ERR_UNSUPPORTED;
    return aligned(p->free, 4) && aligned(p->counts, 4) ? CBS_OK : CBS_ERR_UNSUPPORTED;
}
int check_pages_sizes(int64_t batch, int64_t tokens, int64_t table_width) {
    if (batch < 0 || tokens < 0 || table_width < 0) return CBS_ERR_INVALID_ARG;
    return batch > 65536 || tokens > (1 << 30) || table_width > INT32_MAX ? CBS_ERR_UNSUPPORTED : CBS_OK;
}
bool all_disjoint(const Span *s, int n) {
    for (int i = 0; i < n; ++i)
        for (int j = 0; j < i; ++j)
            if (!disjoint(s[i], {s[j]})) return false;
    return true;
}

}  // namespace

extern "C" {

int cbs_add_rms_norm(conv_bn_silu_t h, const void *x, int64_t x_stride, const void *residual, int64_t residual_stride,
                     int residual_dtype, const void *weight, int weight_dtype, float eps, void *sum, int64_t sum_stride,
                     void *y, int y_dtype, int64_t M, int64_t K, int dtype, void *stream) {
    if (!handle_live(h)) return CBS_ERR_BAD_HANDLE;
    if (!value_type(dtype) || (y_dtype != dtype && y_dtype != CBS_DTYPE_I8)) return CBS_ERR_INVALID_ARG;
    if (M < 0 || K < 1 || !std::isfinite(eps) || eps < 0x1p-126f) return CBS_ERR_INVALID_ARG;
    if (residual && residual_dtype != dtype && residual_dtype != CBS_DTYPE_F32) return CBS_ERR_INVALID_ARG;
    if (weight && weight_dtype != dtype && weight_dtype != CBS_DTYPE_F32) return CBS_ERR_INVALID_ARG;
    if (M > kMaxRows || K > kMaxK) return CBS_ERR_UNSUPPORTED;
    if (M == 0) return CBS_OK;
    if (!x || !y || x_stride < K || (residual != nullptr) != (sum != nullptr)) return CBS_ERR_INVALID_ARG;
    if (residual && (residual_stride < K || sum_stride < K)) return CBS_ERR_INVALID_ARG;
    if (x_stride > kMaxStride || (residual && (residual_stride > kMaxStride || sum_stride > kMaxStride)))
        return CBS_ERR_UNSUPPORTED;
    const bool int8 = y_dtype == CBS_DTYPE_I8;
    const int64_t e = element(dtype), er = element(residual_dtype);
    const auto rows = [&](const void *p, int64_t stride, int64_t size) { return span(p, ((M - 1) * stride + K) * size); };
    const Span sx = rows(x, x_stride, e), sr = rows(residual, residual_stride, er), ss = rows(sum, sum_stride, er);
    const Span sw = span(weight, K * element(weight_dtype)), sy = span(y, int8 ? cbs::rows8_bytes(M, K) : M * K * e);
    const bool in_place = residual && sum == residual && (sum_stride == residual_stride || M == 1);
    if (!disjoint(sy, {sx, sr, ss, sw}) || !disjoint(ss, {sx, sw}) || (!in_place && !disjoint(ss, {sr})))
        return CBS_ERR_INVALID_ARG;
    if (!aligned(x, e) || !aligned(y, int8 ? 16 : e) || (weight && !aligned(weight, element(weight_dtype))) ||
        (residual && (!aligned(residual, er) || !aligned(sum, er))))
        return CBS_ERR_UNSUPPORTED;
    const int rc = check_device(h);
    if (rc != CBS_OK) return rc;
    (void)hipGetLastError();
    const NormArgs a{x, x_stride, residual, residual_stride, weight, sum, sum_stride, y, (int)M, (int)K, dtype,
                     residual_dtype, weight_dtype, int8, eps};
    return record_hip(launch_add_rms_norm(a, (hipStream_t)stream));
}

int cbs_rotary_apply(conv_bn_silu_t h, const cbs_rotary *rotary, const void *x, int64_t token_stride,
                     int64_t head_stride, const int32_t *positions, int64_t tokens, int heads, int dim, int dtype,
                     void *out, int64_t out_token_stride, int64_t out_head_stride, void *stream) {
    if (!handle_live(h)) return CBS_ERR_BAD_HANDLE;
    if (!value_type(dtype) || tokens < 0 || heads < 1 || dim < 1) return CBS_ERR_INVALID_ARG;
    int rc = check_rotary(rotary, dim);
    if (rc != CBS_OK) return rc;
    if (dim > kMaxDim || heads > kMaxHeads || tokens > INT32_MAX / heads) return CBS_ERR_UNSUPPORTED;
    if (tokens == 0) return CBS_OK;
    if (!x || !out || !positions) return CBS_ERR_INVALID_ARG;
    rc = check_strides(tokens, heads, dim, token_stride, head_stride);
    if (rc == CBS_OK) rc = check_strides(tokens, heads, dim, out_token_stride, out_head_stride);
    if (rc != CBS_OK) return rc;
    const int64_t e = element(dtype);
    const Heads from{x, token_stride, head_stride, tokens, heads, dim, e};
    const Heads to{out, out_token_stride, out_head_stride, tokens, heads, dim, e};
    const Span sp = span(positions, tokens * 4);
    if (!to.apart() || (!to.same(from) && !to.beside(from)) || !disjoint(to.all(), {sp, frequencies_of(*rotary)}))
        return CBS_ERR_INVALID_ARG;
    if (!aligned(x, e) || !aligned(out, e) || !aligned(positions, 4)) return CBS_ERR_UNSUPPORTED;
    rc = check_device(h);
    if (rc != CBS_OK) return rc;
    (void)hipGetLastError();
    const RotaryArgs a{*rotary, x, nullptr, nullptr, token_stride, head_stride, 0, 0, 0, 0, out_token_stride,
                       out_head_stride, out, cbs_paged_cache{}, positions, nullptr, tokens, heads, 0, dim, dtype};
    return record_hip(launch_rotary(a, (hipStream_t)stream));
}

int cbs_rotary_cache_write(conv_bn_silu_t h, const cbs_rotary *rotary, const cbs_paged_cache *cache, const void *q,
                           int64_t q_token_stride, int64_t q_head_stride, const void *k, int64_t k_token_stride,
                           int64_t k_head_stride, const void *v, int64_t v_token_stride, int64_t v_head_stride,
                           const int32_t *positions, const int32_t *slots, int64_t tokens, int heads, int dtype,
                           void *q_out, int64_t out_token_stride, int64_t out_head_stride, void *stream) {
    if (!handle_live(h)) return CBS_ERR_BAD_HANDLE;
    int rc = check_cache(cache);
    if (rc != CBS_OK) return rc;
    if (!value_type(dtype) || tokens < 0 || heads < 0) return CBS_ERR_INVALID_ARG;
    rc = check_rotary(rotary, cache->dim);
    if (rc != CBS_OK) return rc;
    if (heads > kMaxHeads || tokens > INT32_MAX / ((int64_t)heads + 2 * cache->heads)) return CBS_ERR_UNSUPPORTED;
    if (tokens == 0) return CBS_OK;
    if (!k || !v || !positions || !slots || (heads > 0 && (!q || !q_out)) || !tensors_disjoint(*cache))
        return CBS_ERR_INVALID_ARG;
    const int64_t e = element(dtype), dim = cache->dim;
    const Heads fk{k, k_token_stride, k_head_stride, tokens, cache->heads, dim, e};
    const Heads fv{v, v_token_stride, v_head_stride, tokens, cache->heads, dim, e};
    const Heads fq{q, q_token_stride, q_head_stride, tokens, heads, dim, e};
    const Heads to{q_out, out_token_stride, out_head_stride, tokens, heads, dim, e};
    for (const Heads *t : {&fk, &fv, &fq, &to}) {
        if (t->heads == 0) continue;
        rc = check_strides(tokens, t->heads, dim, t->token, t->head);
        if (rc != CBS_OK) return rc;
    }
    const Span sp = span(positions, tokens * 4), ss = span(slots, tokens * 4), sf = frequencies_of(*rotary);
    for (const Span &s : {fk.all(), fv.all(), sp, ss, sf})
        if (!clear_of_cache(s, *cache)) return CBS_ERR_INVALID_ARG;
    if (heads > 0) {
        if (!clear_of_cache(fq.all(), *cache) || !clear_of_cache(to.all(), *cache)) return CBS_ERR_INVALID_ARG;
        if (!to.apart() || (!to.same(fq) && !to.beside(fq)) || !to.beside(fk) || !to.beside(fv) ||
            !disjoint(to.all(), {sp, ss, sf}))
            return CBS_ERR_INVALID_ARG;
        if (!aligned(q, e) || !aligned(q_out, e)) return CBS_ERR_UNSUPPORTED;
    }
    if (!aligned(k, e) || !aligned(v, e) || !aligned(positions, 4) || !aligned(slots, 4)) return CBS_ERR_UNSUPPORTED;
    rc = check_device(h);
    if (rc != CBS_OK) return rc;
    (void)hipGetLastError();
    const RotaryArgs a{*rotary, q, k, v, q_token_stride, q_head_stride, k_token_stride, k_head_stride, v_token_stride,
                       v_head_stride, out_token_stride, out_head_stride, q_out, *cache, positions, slots, tokens, heads,
                       cache->heads, cache->dim, dtype};
    return record_hip(launch_rotary(a, (hipStream_t)stream));
}

int64_t cbs_grow_pages_workspace(int64_t batch, int64_t tokens) {
    return check_pages_sizes(batch, tokens, 0) == CBS_OK ? grow_workspace(batch, tokens) : -1;
}
int64_t cbs_release_pages_workspace(int64_t batch, int64_t table_width) {
    return check_pages_sizes(batch, 0, table_width) == CBS_OK ? release_workspace(batch, table_width) : -1;
}

int cbs_grow_pages(conv_bn_silu_t h, const cbs_page_pool *pool, int32_t *table, int64_t table_stride,
                   int64_t table_width, int32_t *lens, const int32_t *more, int64_t batch, int64_t tokens,
                   int32_t *starts, int32_t *slots, int32_t *positions, void *workspace, int64_t workspace_bytes,
                   void *stream) {
    if (!handle_live(h)) return CBS_ERR_BAD_HANDLE;
    int rc = check_pool(pool);
    if (rc == CBS_OK) rc = check_pages_sizes(batch, tokens, table_width);
    if (rc != CBS_OK) return rc;
    if (!starts || (batch > 0 && (!lens || !more || (!table && table_width > 0) || table_stride < table_width)) ||
        (tokens > 0 && (!slots || !positions)))
        return CBS_ERR_INVALID_ARG;
    if (table_stride > kMaxStride) return CBS_ERR_UNSUPPORTED;
    const int64_t need = grow_workspace(batch, tokens);
    if (need > 0 && (!workspace || workspace_bytes < need)) return CBS_ERR_INVALID_ARG;
    const Span all[] = {span(pool->free, pool->pages * 4), span(pool->counts, 12),
                        span(table, batch > 0 ? ((batch - 1) * table_stride + table_width) * 4 : 0), span(lens, batch * 4),
                        span(more, batch * 4), span(starts, (batch + 1) * 4), span(slots, tokens * 4),
                        span(positions, tokens * 4), span(workspace, need)};
    if (!all_disjoint(all, 9)) return CBS_ERR_INVALID_ARG;
    for (const int32_t *p : {(const int32_t *)table, (const int32_t *)lens, more, (const int32_t *)starts,
                             (const int32_t *)slots, (const int32_t *)positions})
        if (!aligned(p, 4)) return CBS_ERR_UNSUPPORTED;
    if (!aligned(workspace, 16)) return CBS_ERR_UNSUPPORTED;
    rc = check_device(h);
    if (rc != CBS_OK) return rc;
    (void)hipGetLastError();
    const PagesArgs a{*pool, table, table_stride, table_width, lens, more, (int)batch, (int)tokens, starts, slots,
                      positions, workspace};
    return record_hip(launch_grow_pages(a, (hipStream_t)stream));
}

int cbs_release_pages(conv_bn_silu_t h, const cbs_page_pool *pool, int32_t *table, int64_t table_stride,
                      int64_t table_width, int32_t *lens, const int32_t *keep, int64_t batch, void *workspace,
                      int64_t workspace_bytes, void *stream) {
    if (!handle_live(h)) return CBS_ERR_BAD_HANDLE;
    int rc = check_pool(pool);
    if (rc == CBS_OK) rc = check_pages_sizes(batch, 0, table_width);
    if (rc != CBS_OK) return rc;
    if (batch == 0) return CBS_OK;
    if (!lens || !keep || (!table && table_width > 0) || table_stride < table_width) return CBS_ERR_INVALID_ARG;
    if (table_stride > kMaxStride) return CBS_ERR_UNSUPPORTED;
    const int64_t need = release_workspace(batch, table_width);
    if (need > 0 && (!workspace || workspace_bytes < need)) return CBS_ERR_INVALID_ARG;
    const Span all[] = {span(pool->free, pool->pages * 4), span(pool->counts, 12),
                        span(table, ((batch - 1) * table_stride + table_width) * 4), span(lens, batch * 4),
                        span(keep, batch * 4), span(workspace, need)};
    if (!all_disjoint(all, 6)) return CBS_ERR_INVALID_ARG;
    for (const int32_t *p : {(const int32_t *)table, (const int32_t *)lens, keep})
        if (!aligned(p, 4)) return CBS_ERR_UNSUPPORTED;
    if (!aligned(workspace, 16)) return CBS_ERR_UNSUPPORTED;
    rc = check_device(h);
    if (rc != CBS_OK) return rc;
    (void)hipGetLastError();
    const PagesArgs a{*pool, table, table_stride, table_width, lens, keep, (int)batch, 0, nullptr, nullptr, nullptr,
                      workspace};
    return record_hip(launch_release_pages(a, (hipStream_t)stream));
}

}  // extern "C"
