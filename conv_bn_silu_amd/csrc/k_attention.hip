// k_attention.hip -- attention of each sequence's newest tokens over its paged
// cache: how a call is divided between the kernels, and the joining of chunks.
#include <hip/hip_runtime.h>

#include "b8_attention.h"

namespace cbs {
namespace {

constexpr int kThreads = 256;

// One row: its chunks' parts, brought to one maximum and added.  A wave to a row.
template <typename T>
__device__ __forceinline__ void join(const AttentionPlan &p, const AttentionPart &part, int64_t line, int n, int64_t out) {
    const int lane = (int)threadIdx.x % 64, dim = p.a.cache.dim;
    const float *ml = part.ml + 2 * line * part.chunks, *o = part.o + line * part.chunks * dim;
    float top = -INFINITY;
    for (int c = 0; c < n; ++c) top = fmaxf(top, ml[2 * c]);
    float sum = 0.f, v[4] = {0.f, 0.f, 0.f, 0.f};
    for (int c = 0; c < n; ++c) {
        const float f = ml[2 * c] == top ? 1.f : __builtin_amdgcn_exp2f(ml[2 * c] - top);
        sum += ml[2 * c + 1] * f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (64 * i + lane < dim) v[i] += o[(int64_t)c * dim + 64 * i + lane] * f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (64 * i + lane < dim) Value<T>::store1((T *)p.a.out + out * dim + 64 * i + lane, divide(v[i], sum));
}

// A workgroup to a sequence and key/value head.
template <typename T> __global__ __launch_bounds__(kThreads) void join_few(const AttentionPlan p) {
    const int kvh = (int)blockIdx.x % p.a.cache.heads, wave = (int)threadIdx.x / 64;
    const Sequence s = sequence(p, (int)blockIdx.x / p.a.cache.heads);
    const int rows = s.n * (int)p.group.d;
    if (is_many(p, rows)) return;
    for (int r = wave; r < rows; r += kThreads / 64) {
        const int r0 = r / p.few.tile * p.few.tile;
        const int n = chunks_of(p.few, keys_of(p, s, r0, min(rows, r0 + p.few.tile)));
        if (n > 1) join<T>(p, p.few, few_line(p, s, kvh, r), n, out_line(p, s, kvh, r));
    }
}

int64_t part_floats(const AttentionPart &part, int64_t lines, int64_t dim) {
    return part.chunks > 1 ? lines * part.chunks * (dim + 2) : 0;
}

struct Sizes {
    int64_t batch, tokens, heads, kv_heads, dim, page_size, table_width;
};
// The division of a call, and the floats of workspace that it takes.
int64_t make_plan(AttentionPlan &p, const Sizes &z, int num_cu) {
    const int64_t group = z.heads / z.kv_heads, limit = z.table_width * z.page_size;
    // 32 rows only where single tokens do not fill 16: the registers they take cost waves
    p.few.tile = z.dim <= 128 && (z.tokens > z.batch || group > 16) ? 32 : 16;
    p.few_only = true;
    const int64_t pairs = z.batch * z.kv_heads;
    // up to 1024 keys a second kernel to join chunks costs more than the other CUs save
    p.few.chunk = (int)(limit <= 1024 ? 1024 : 2048);
    if (limit > 1024) {
        const int64_t even = limit * pairs / (16 * num_cu) / 256 * 256;
        p.few.chunk = (int)(even < 512 ? 512 : even > 1024 ? 1024 : even);
    }
    p.few.chunks = (int)((limit + p.few.chunk - 1) / p.few.chunk);
    if (p.few.chunks < 1) p.few.chunks = 1;
    const int64_t few_lines = p.few_only ? z.tokens * z.heads : pairs * p.few.tile;
    p.few.o = nullptr;
    p.few.ml = p.few.o + few_lines * p.few.chunks * z.dim;
    return part_floats(p.few, few_lines, z.dim);
}

}  // namespace

int64_t attention_workspace(int num_cu, int64_t batch, int64_t tokens, int heads, int kv_heads, int dim, int page_size,
                            int64_t table_width) {
    AttentionPlan p{};
    return 4 * make_plan(p, Sizes{batch, tokens, heads, kv_heads, dim, page_size, table_width}, num_cu);
}

hipError_t launch_paged_attention(const AttentionArgs &a, int num_cu, hipStream_t st) {
    AttentionPlan p{};
    p.a = a;
    p.page = make_fastdiv((uint32_t)a.cache.page_size);
    p.group = make_fastdiv((uint32_t)(a.heads / a.cache.heads));
    make_plan(p, Sizes{a.batch, a.tokens, a.heads, a.cache.heads, a.cache.dim, a.cache.page_size, a.table_width}, num_cu);
    float *const ws = (float *)a.workspace;
    const int64_t few_ml = p.few.ml - p.few.o;
    p.few.o = ws, p.few.ml = ws + few_ml;
    hipError_t e = launch_attend_few(p, st);
    if (e != hipSuccess || p.few.chunks == 1) return e;
    const unsigned grid = (unsigned)(a.batch * a.cache.heads);
    if (a.dtype == CBS_DTYPE_BF16) join_few<__bf16><<<grid, kThreads, 0, st>>>(p);
    else join_few<_Float16><<<grid, kThreads, 0, st>>>(p);
    return hipGetLastError();
}

}  // namespace cbs
