// st_launch.h -- host-side entry points of the kernel files of cbs_step.h's operators, used by
// st_api.cpp, which has validated every argument.  Each launcher enqueues its kernels and
// returns the launch's error.
#pragma once

#include "../../include/cbs_step.h"
#include "b8_launch.h"

namespace cbs {

struct NormArgs {
    const void *x;
    int64_t x_stride;
    const void *residual;  // or null
    int64_t residual_stride;
    const void *weight;  // or null
    void *sum;
    int64_t sum_stride;
    void *y;  // values, or a buffer of rows in 8 bits
    int M, K, dtype, residual_dtype, weight_dtype;
    bool int8;
    float eps;
};
hipError_t launch_add_rms_norm(const NormArgs &a, hipStream_t st);

struct RotaryArgs {
    cbs_rotary rotary;
    const void *q, *k, *v;  // k and v null without a cache
    int64_t q_token, q_head, k_token, k_head, v_token, v_head, out_token, out_head;
    void *q_out;
    cbs_paged_cache cache;
    const int32_t *positions, *slots;
    int64_t tokens;
    int heads, kv_heads, dim, dtype;  // kv_heads 0 without a cache
};
hipError_t launch_rotary(const RotaryArgs &a, hipStream_t st);

struct PagesArgs {
    cbs_page_pool pool;
    int32_t *table;
    int64_t table_stride, table_width;
    int32_t *lens;
    const int32_t *change;  // new tokens, or tokens to keep
    int batch, tokens;
    int32_t *starts, *slots, *positions;
    void *workspace;
};
int64_t grow_workspace(int64_t batch, int64_t tokens);
int64_t release_workspace(int64_t batch, int64_t table_width);
hipError_t launch_grow_pages(const PagesArgs &a, hipStream_t st);
hipError_t launch_release_pages(const PagesArgs &a, hipStream_t st);

}  // namespace cbs
