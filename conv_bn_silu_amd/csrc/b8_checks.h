// b8_checks.h -- host-side checks of arguments that the entry points of b8_api.cpp and
// st_api.cpp share.
#pragma once

#include <climits>
#include <cstdint>
#include <initializer_list>

#include "../../include/cbs_block8.h"

namespace cbs {

constexpr int64_t kMaxStride = 1ll << 40;  // keeps 64-bit offsets exact

struct Span {
    uintptr_t lo, hi;  // [lo, hi)
};
inline Span span(const void *p, int64_t bytes) { return {(uintptr_t)p, (uintptr_t)p + (uintptr_t)(p ? bytes : 0)}; }
inline bool disjoint(Span a, std::initializer_list<Span> others) {
    for (const Span &o : others)
        if (a.lo < o.hi && o.lo < a.hi) return false;
    return true;
}

inline bool value_type(int dtype) { return dtype == CBS_DTYPE_F32 || dtype == CBS_DTYPE_BF16 || dtype == CBS_DTYPE_F16; }
inline int64_t element(int dtype) { return dtype == CBS_DTYPE_F32 ? 4 : dtype == CBS_DTYPE_I8 ? 1 : 2; }
inline bool aligned(const void *p, int64_t to) { return (uintptr_t)p % (uintptr_t)to == 0; }

// The cache's own fields; its bytes and the spans of its tensors.
inline int check_cache(const cbs_paged_cache *c) {
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
inline int64_t cache_rows(const cbs_paged_cache &c) { return c.pages * c.heads * c.page_size; }
inline int64_t cache_bytes(const cbs_paged_cache &c) { return cache_rows(c) * c.dim * element(c.dtype); }
inline bool clear_of_cache(Span s, const cbs_paged_cache &c) {
    return disjoint(s, {span(c.k, cache_bytes(c)), span(c.v, cache_bytes(c)), span(c.k_scale, cache_rows(c) * 4),
                        span(c.v_scale, cache_rows(c) * 4)});
}
inline bool tensors_disjoint(const cbs_paged_cache &c) {
    const Span k = span(c.k, cache_bytes(c)), v = span(c.v, cache_bytes(c));
    const Span ks = span(c.k_scale, cache_rows(c) * 4), vs = span(c.v_scale, cache_rows(c) * 4);
    return disjoint(k, {v, ks, vs}) && disjoint(v, {ks, vs}) && disjoint(ks, {vs});
}

inline int check_strides(int64_t tokens, int64_t heads, int64_t dim, int64_t token_stride, int64_t head_stride) {
    (void)tokens;
    if (head_stride < dim && heads > 1) return CBS_ERR_INVALID_ARG;
    if (token_stride < dim && tokens > 1) return CBS_ERR_INVALID_ARG;
    if (token_stride < 0 || head_stride < 0) return CBS_ERR_INVALID_ARG;
    if (token_stride > kMaxStride || head_stride > kMaxStride) return CBS_ERR_UNSUPPORTED;
    return CBS_OK;
}
inline int64_t strided_bytes(int64_t tokens, int64_t heads, int64_t dim, int64_t token_stride, int64_t head_stride, int dtype) {
    return ((tokens - 1) * token_stride + (heads - 1) * head_stride + dim) * element(dtype);
}

}  // namespace cbs
