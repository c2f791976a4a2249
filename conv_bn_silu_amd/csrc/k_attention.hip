// k_attention.hip -- attention of each sequence's newest tokens over its paged
// cache: how a call is divided between the kernels, and the joining of chunks.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "b8_attention.h"

namespace cbs {
namespace {

constexpr int kWaves = 4, kThreads = 64 * kWaves;

// One row: its chunks' parts, brought to one maximum and added.  A wave to a row: its
// lanes are the chunks where maxima and sums are concerned, and the dims for the outputs,
// whose loads for 8 chunks at a time do not wait for each other.
template <typename T, int ND>
__device__ __forceinline__ void join_dims(const AttentionPlan &p, const AttentionPart &part, int64_t line, int n, int64_t out) {
    const int lane = (int)threadIdx.x % 64, dim = p.a.cache.dim;
    const float *ml = part.ml + 2 * line * part.room, *o = part.o + line * part.room * dim;
    float top = -INFINITY;
    for (int c = lane; c < n; c += 64) top = fmaxf(top, ml[2 * c]);
#pragma unroll
    for (int x = 1; x < 64; x *= 2) top = fmaxf(top, __shfl_xor(top, x, 64));
    float sum = 0.f, v[ND] = {};
    for (int c0 = 0; c0 < n; c0 += 64) {
        float f = 0.f, l = 0.f;
        if (c0 + lane < n) {
            const float m = ml[2 * (c0 + lane)];
            f = m == top ? 1.f : __builtin_amdgcn_exp2f(m - top);
            l = ml[2 * (c0 + lane) + 1] * f;
        }
#pragma unroll
        for (int x = 1; x < 64; x *= 2) l += __shfl_xor(l, x, 64);
        sum += l;
        const int n0 = min(64, n - c0);
        for (int c = 0; c < n0; c += 8) {
            float part_o[8][ND];
#pragma unroll
            for (int e = 0; e < 8; ++e)
#pragma unroll
                for (int i = 0; i < ND; ++i)
                    part_o[e][i] = o[(int64_t)(c0 + min(c + e, n0 - 1)) * dim + min(64 * i + lane, dim - 1)];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float w = __shfl(f, min(c + e, 63), 64);
#pragma unroll
                for (int i = 0; i < ND; ++i)
                    if (c + e < n0) v[i] += part_o[e][i] * w;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < ND; ++i)
        if (64 * i + lane < dim) Value<T>::store1((T *)p.a.out + out * dim + 64 * i + lane, divide(v[i], sum));
}

template <typename T>
__device__ __forceinline__ void join(const AttentionPlan &p, const AttentionPart &part, int64_t line, int n, int64_t out) {
    if (p.a.cache.dim <= 128) join_dims<T, 2>(p, part, line, n, out);
    else join_dims<T, 4>(p, part, line, n, out);
}

// A wave to a row of a sequence and key/value head; beside attend_many, there is at most a tile of them.
template <typename T> __device__ __forceinline__ void join_few(const AttentionPlan &p, int at) {
    const int per = (p.few.tile + kWaves - 1) / kWaves, pair = at / per, wave = (int)threadIdx.x / 64;
    const int kvh = pair % p.a.cache.heads;
    const Sequence s = sequence(p, pair / p.a.cache.heads);
    const int rows = s.n * (int)p.group.d;
    if (is_many(p, rows)) return;
    for (int r = at % per * kWaves + wave; r < rows; r += per * kWaves) {
        const int r0 = r / p.few.tile * p.few.tile;
        const int n = chunks_of(p.few, keys_of(p, s, r0, min(rows, r0 + p.few.tile)));
        if (n > 1) join<T>(p, p.few, few_line(p, s, kvh, r), n, out_line(p, s, kvh, r));
    }
}

// A wave to a row of the output.
template <typename T> __device__ __forceinline__ void join_many(const AttentionPlan &p, int at) {
    const int lane = (int)threadIdx.x % 64;
    const int64_t line = (int64_t)at * kWaves + threadIdx.x / 64;
    if (line >= (int64_t)p.a.tokens * p.a.heads) return;
    const int token = (int)(line / p.a.heads), head = (int)(line - (int64_t)token * p.a.heads);
    const int kvh = (int)p.group.div((uint32_t)head);
    for (int b0 = 0; b0 < p.a.batch; b0 += 64) {
        Sequence s{0, 0, 0, 0};
        if (b0 + lane < p.a.batch) s = sequence(p, b0 + lane);
        const uint64_t mine = __ballot(s.first <= token && token < s.first + s.n);
        if (!mine) continue;
        s = sequence(p, b0 + __builtin_ctzll(mine));
        const int rows = s.n * (int)p.group.d, r = (token - s.first) * (int)p.group.d + head - kvh * (int)p.group.d;
        if (!is_many(p, rows)) return;
        const int r0 = r / p.many.tile * p.many.tile;
        const int n = chunks_of(p.many, keys_of(p, s, r0, min(rows, r0 + p.many.tile)));
        if (n > 1) join<T>(p, p.many, line, n, line);
        return;
    }
}

// The first `few` workgroups have attend_few's rows, the others attend_many's.
template <typename T> __global__ __launch_bounds__(kThreads) void join_parts(const AttentionPlan p, int few) {
    if ((int)blockIdx.x < few) join_few<T>(p, (int)blockIdx.x);
    else join_many<T>(p, (int)blockIdx.x - few);
}

int64_t round_up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }
// Lays a kernel's parts out in the workspace, `at` floats of which are taken.
void place_parts(AttentionPart &part, float *ws, int64_t &at, int64_t lines, int64_t dim) {
    if (part.room <= 1) return;
    part.o = ws + at;
    at += lines * part.room * dim;
    part.ml = ws + at;
    at += lines * part.room * 2;
}

// The division of a call; returns the bytes of workspace that it takes.
int64_t make_plan(AttentionPlan &p, int64_t batch, int64_t tokens, int64_t heads, int64_t kv_heads, int64_t dim,
                  int64_t page_size, int64_t table_width, int64_t num_cu, float *ws) {
    const int64_t group = heads / kv_heads, limit = table_width * page_size, pairs = batch * kv_heads;
    // 32 rows only where the average sequence has more than 16: the registers they take cost
    // waves (8 sequences of 2 tokens, groups of 4, over 3000 keys: 41 us, with 16 rows 25)
    p.few.tile = dim <= 128 && tokens * group > 16 * batch ? 32 : 16;
    // With no more tokens than sequences they are single tokens, as a rule, and a launch of attend_many that
    // finds nothing would cost 4 of 10 us.  A batch padded with empty sequences breaks the rule, and its chunk
    // goes 32 rows at a time (60 tokens after 4000, 32 heads over 8, us: alone 28, with 58 empty sequences beside
    // it, which still is attend_many, 52, with 63 269).
    p.few_only = tokens <= batch || tokens * group <= p.few.tile;
    // Two waves to a row where tiles of 256 rows leave CUs idle and a tile's keys are not many times
    // its tokens (then chunks fill the CUs as well).  One and two, us: a prompt of 1000 49.4 and
    // 36.0, of 2000 85.1 and 73.0, of 4000 167 and 211; 512 tokens after 4000 36.4 and 38.5.  In
    // between it goes both ways: three of 200 to 900 after up to 3000, 15 heads over 3, 73 and 62;
    // 2000 after 8000, 4 heads over 1, 72.5 and 77.9.
    const int64_t partial = std::min(batch, tokens * group / (p.few.tile + 1));
    const int64_t keys = p.a.window ? std::min(limit, p.a.window + tokens / std::max<int64_t>(1, batch)) : limit;
    p.split = dim <= 128 && (2 * tokens * group / many_tile(dim, true, false) + partial) * kv_heads < 2 * num_cu && keys * batch <= 8 * tokens;
    p.many.tile = many_tile(dim, p.a.cache.dtype == CBS_DTYPE_I8, p.split);
    p.slots = (int)(tokens * group / p.many.tile + partial);

    // attend_few: 1024 keys are soon read, and joining chunks takes a kernel more.  Beyond,
    // so many chunks that every CU has several workgroups to its name, but no more than
    // that: a workgroup needs some steps to fill its pipe.  The table's width is all that is
    // known of the lengths; where it leaves room for far more, larger chunks keep the
    // workgroups that find nothing to do below 16384.
    const int64_t even = limit * pairs / (16 * num_cu) / 256 * 256, wide = std::min<int64_t>(1 << 30, round_up(limit * pairs / 16384, 256));
    p.few.chunk = limit <= 1024 ? 1024 : (int)std::max(wide, std::min<int64_t>(2048, std::max<int64_t>(512, even)));
    p.few.chunks = p.few.room = (int)std::max<int64_t>(1, (limit + p.few.chunk - 1) / p.few.chunk);

    // attend_many: chunks only where there are too few tiles for the CUs, and no more
    // workgroups than CUs, each of which holds one (512 tokens after 4000, 8 heads over 2: 162
    // workgroups 43 us, 252 40, 324 54).  Of the tiles that may be partial, half count.
    // The workspace has room for the chunks of either form (it is asked for without the window),
    // by the tiles of 8-bit caches.
    p.many.room = 1;
    for (int split = dim <= 128; split >= 0; --split) {
        const int64_t groups2 = std::max<int64_t>(1, (2 * tokens * group / many_tile(dim, true, split) + partial) * kv_heads);
        const int64_t want = limit <= 512 ? 1 : std::max<int64_t>(1, 2 * num_cu / groups2);
        const int chunk = want == 1 ? 1 << 30 : (int)std::max<int64_t>(256, round_up((limit + want - 1) / want, 64));
        const int chunks = want == 1 ? 1 : (int)std::max<int64_t>(1, (limit + chunk - 1) / chunk);
        p.many.room = std::max(p.many.room, chunks);
        if (split == (int)p.split) p.many.chunk = chunk, p.many.chunks = chunks;
    }

    int64_t at = 0;
    place_parts(p.few, ws, at, p.few_only ? tokens * heads : pairs * p.few.tile, dim);
    if (!p.few_only) place_parts(p.many, ws, at, tokens * heads, dim);
    return 4 * at;
}

template <typename T> hipError_t launch_joins(const AttentionPlan &p, hipStream_t st) {
    const int64_t lines = !p.few_only && p.many.chunks > 1 ? (int64_t)p.a.tokens * p.a.heads : 0;
    const int64_t many = (lines + kWaves - 1) / kWaves;
    const int64_t few = p.few.chunks > 1 ? (int64_t)p.a.batch * p.a.cache.heads * ((p.few.tile + kWaves - 1) / kWaves) : 0;
    if (few + many > 0) join_parts<T><<<(unsigned)(few + many), kThreads, 0, st>>>(p, (int)few);
    return hipGetLastError();
}

}  // namespace

int64_t attention_workspace(int num_cu, int64_t batch, int64_t tokens, int heads, int kv_heads, int dim, int page_size,
                            int64_t table_width) {
    AttentionPlan p{};
    return make_plan(p, batch, tokens, heads, kv_heads, dim, page_size, table_width, num_cu, nullptr);
}

hipError_t launch_paged_attention(const AttentionArgs &a, int num_cu, hipStream_t st) {
    AttentionPlan p{};
    p.a = a;
    p.page = make_fastdiv((uint32_t)a.cache.page_size);
    p.group = make_fastdiv((uint32_t)(a.heads / a.cache.heads));
    make_plan(p, a.batch, a.tokens, a.heads, a.cache.heads, a.cache.dim, a.cache.page_size, a.table_width, num_cu,
              (float *)a.workspace);
    hipError_t e = launch_attend_few(p, st);
    if (e == hipSuccess && !p.few_only) e = launch_attend_many(p, st);
    if (e != hipSuccess) return e;
    return a.dtype == CBS_DTYPE_BF16 ? launch_joins<__bf16>(p, st) : launch_joins<_Float16>(p, st);
}

}  // namespace cbs
