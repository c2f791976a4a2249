// b8_launch.h -- host-side entry points of the kernel files of the 8-bit block
// operators, used by b8_api.cpp, which has validated every argument.  Each
// launcher enqueues its kernels and returns the launch's error.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/cbs_block8.h"

namespace cbs {

// Division by a divisor fixed for the launch, exact for numerators below 2^31:
// n / d = (n * mul) >> shift with shift = 31 + ceil(log2 d) and
// mul = ceil(2^shift / d) < 2^32 (the excess mul * d - 2^shift < d <= 2^(shift - 31),
// times n < 2^31, stays below 2^shift).
struct FastDiv {
    uint32_t d, mul, shift;
#ifdef __HIPCC__
    __host__ __device__ __forceinline__
#else
    inline
#endif
    uint32_t div(uint32_t n) const { return (uint32_t)(((uint64_t)n * mul) >> shift); }
};
inline FastDiv make_fastdiv(uint32_t d) {
    uint32_t l = 0;
    while ((1ull << l) < d) ++l;
    const uint32_t shift = 31 + l;
    return FastDiv{d, (uint32_t)(((1ull << shift) + d - 1) / d), shift};
}

struct LinearArgs {
    const void *x;
    int64_t x_stride;
    const int8_t *w;
    const float *w_scale, *bias;  // bias may be null
    void *y;
    int M, N, K, dtype, act;
    void *workspace;
    const void *rows;  // in 8 bits already, in place of x; else null
};
int64_t linear_workspace(int64_t M, int64_t N, int64_t K, bool rows);  // rows: given in 8 bits
int64_t rows8_bytes(int64_t M, int64_t K);
hipError_t launch_int8_linear(const LinearArgs &a, hipStream_t st);

struct CacheIo {
    cbs_paged_cache cache;
    const void *k, *v;                  // write: sources
    int64_t k_token, k_head, v_token, v_head;
    void *k_out, *v_out;                // read: destinations
    const int32_t *slots;
    int64_t tokens;
    int dtype;
};
hipError_t launch_cache_write(const CacheIo &a, hipStream_t st);
hipError_t launch_cache_read(const CacheIo &a, hipStream_t st);

struct AttentionArgs {
    const void *q;
    int64_t q_token, q_head;
    cbs_paged_cache cache;
    const int32_t *table;
    int64_t table_stride;
    int table_width;
    const int32_t *starts, *lens;
    int batch, tokens, heads, window;
    float scale;
    void *out;
    int dtype;
    void *workspace;
};
int64_t attention_workspace(int num_cu, int64_t batch, int64_t tokens, int heads, int kv_heads, int dim, int page_size,
                            int64_t table_width);
hipError_t launch_paged_attention(const AttentionArgs &a, int num_cu, hipStream_t st);

}  // namespace cbs
