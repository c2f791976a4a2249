// k_attention.hip -- attention of each sequence's newest tokens over its paged
// cache.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "b8_device.h"
#include "b8_launch.h"

namespace cbs {
namespace {

constexpr int kThreads = 256;

struct Params {
    AttentionArgs a;
    FastDiv page;
    int group;
};

template <typename C> __device__ __forceinline__ f32x8 cache8(const C *p, float s) {
    if constexpr (std::is_same_v<C, int8_t>) {
        const u32x2 c = *(const u32x2 *)p;
        f32x8 x;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = (float)(int8_t)(c[i / 4] >> (8 * (i % 4))) * s;
        return x;
    } else {
        return Value<C>::load8(p);
    }
}

__device__ __forceinline__ float block_reduce(float v, bool is_max, float *tmp) {
#pragma unroll
    for (int o = 1; o < 64; o *= 2) {
        const float w = __shfl_xor(v, o, 64);
        v = is_max ? fmaxf(v, w) : v + w;
    }
    __syncthreads();
    if (threadIdx.x % 64 == 0) tmp[threadIdx.x / 64] = v;
    __syncthreads();
    float r = tmp[0];
    for (int i = 1; i < kThreads / 64; ++i) r = is_max ? fmaxf(r, tmp[i]) : r + tmp[i];
    return r;
}

// One workgroup per query token and head; 256 keys at a time, one a lane, with
// the running maximum and sum of the softmax.
template <typename T, typename C> __global__ __launch_bounds__(kThreads) void attend(const Params p) {
    __shared__ float qs[256], ps[kThreads], tmp[kThreads / 64], part[kThreads / 32][256];
    __shared__ int64_t rows[kThreads];
    const AttentionArgs &a = p.a;
    const int t = (int)threadIdx.x, token = (int)blockIdx.x, head = (int)blockIdx.y, dim = a.cache.dim;
    int b = 0, first = 0, next = 0;
    for (; b < a.batch; ++b) {
        first = max(0, min(a.starts[b], a.tokens));
        next = max(0, min(a.starts[b + 1], a.tokens));
        if (token >= first && token < next) break;
    }
    if (b == a.batch) return;
    const int kv_head = head / p.group;
    const int64_t len = a.lens[b], pos = len - (next - first) + (token - first);
    const int64_t limit = (int64_t)a.table_width * p.page.d;
    const int end = (int)max((int64_t)0, min(min(pos + 1, len), limit));
    const int begin = a.window ? (int)max((int64_t)0, pos + 1 - a.window) : 0;
    for (int d = t; d < dim; d += kThreads)
        qs[d] = Value<T>::load1((const T *)a.q + token * a.q_token + head * a.q_head + d) * a.scale;
    float top = -INFINITY, sum = 0.f;
    const int dc = t % 32 * 8;  // this lane's values of the output, keys t / 32, + 8, ...
    f32x8 o = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int j0 = begin; j0 < end; j0 += kThreads) {
        __syncthreads();
        const int j = j0 + t;
        float s = -INFINITY;
        int64_t row = -1;
        if (j < end) {
            const uint32_t pg = p.page.div((uint32_t)j);
            const int page = a.table[b * a.table_stride + pg];
            if (page >= 0 && page < a.cache.pages) {
                row = ((int64_t)page * a.cache.heads + kv_head) * p.page.d + (j - (int)(pg * p.page.d));
                const float ks = std::is_same_v<C, int8_t> ? a.cache.k_scale[row] : 1.f;
                s = 0.f;
                for (int d = 0; d < dim; d += 8) {
                    const f32x8 k = cache8<C>((const C *)a.cache.k + row * dim + d, ks);
#pragma unroll
                    for (int i = 0; i < 8; ++i) s = __builtin_fmaf(qs[d + i], k[i], s);
                }
            }
        }
        rows[t] = row;
        const float new_top = fmaxf(top, block_reduce(s, true, tmp));
        const float e = row < 0 ? 0.f : __expf(s - new_top);
        ps[t] = e;
        const float fade = new_top == -INFINITY ? 1.f : __expf(top - new_top);
        sum = sum * fade + block_reduce(e, false, tmp);
        top = new_top;
        if (dc < dim) {
            o *= fade;
            for (int i = t / 32; i < kThreads; i += kThreads / 32) {
                const int64_t r = rows[i];
                if (r < 0) continue;
                const float vs = std::is_same_v<C, int8_t> ? a.cache.v_scale[r] : 1.f;
                o += cache8<C>((const C *)a.cache.v + r * dim + dc, vs) * ps[i];
            }
        }
    }
    __syncthreads();
    if (dc < dim)
        for (int i = 0; i < 8; ++i) part[t / 32][dc + i] = o[i];
    __syncthreads();
    for (int d = t; d < dim; d += kThreads) {
        float v = 0.f;
        for (int i = 0; i < kThreads / 32; ++i) v += part[i][d];
        Value<T>::store1((T *)a.out + ((int64_t)token * a.heads + head) * dim + d, sum > 0.f || sum != sum ? v / sum : 0.f);
    }
}

template <typename T> hipError_t launch1(const AttentionArgs &a, hipStream_t st) {
    const Params p{a, make_fastdiv((uint32_t)a.cache.page_size), a.heads / a.cache.heads};
    const dim3 grid(a.tokens, a.heads);
    if (a.cache.dtype == CBS_DTYPE_I8) attend<T, int8_t><<<grid, kThreads, 0, st>>>(p);
    else attend<T, T><<<grid, kThreads, 0, st>>>(p);
    return hipGetLastError();
}

}  // namespace

int64_t attention_workspace(int num_cu, int64_t batch, int64_t tokens, int heads, int kv_heads, int dim, int page_size,
                            int64_t table_width) {
    (void)num_cu, (void)batch, (void)tokens, (void)heads, (void)kv_heads, (void)dim, (void)page_size, (void)table_width;
    return 0;
}

hipError_t launch_paged_attention(const AttentionArgs &a, int num_cu, hipStream_t st) {
    (void)num_cu;
    return a.dtype == CBS_DTYPE_BF16 ? launch1<__bf16>(a, st) : launch1<_Float16>(a, st);
}

}  // namespace cbs
