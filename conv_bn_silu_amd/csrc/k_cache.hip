// k_cache.hip -- the paged key/value cache: rows quantised (or converted) as they
// are written, and read back.
//
// Both directions are copies with a little arithmetic: bound by HBM (per row of
// D values: e D + D + 4 bytes each way for 8-bit caches).  A row belongs to a
// team of 16 lanes (32 when D > 128), 8 elements a lane, so that a lane moves
// one 16-byte piece of a 16-bit row and the row's largest magnitude is a 4-step
// exchange inside the team; a workgroup handles 16 (8) rows and ends: as for the
// plain copy, many short workgroups keep the most bytes in flight.  32768 tokens x 8 heads
// x 128, bf16: written and read back in 88 us, 4.6 TB/s (a large copy: 6.3), of which the write takes
// 57 and the read 36.  One set of tensors over and over, write and read, us: 8-bit cache 46 and 33,
// 16 bits 42 and 41 (6.4 TB/s), 32 bits 80 and 69.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "b8_device.h"
#include "b8_launch.h"

namespace cbs {
namespace {

constexpr int kThreads = 256;

struct CacheParams {
    CacheIo io;
    FastDiv heads, page;
    uint32_t rows;   // tokens * heads of the launch
    uint32_t slots;  // pages * page size
};

// Largest over a team of TEAM consecutive lanes, in every lane of it.
template <int TEAM> __device__ __forceinline__ uint32_t team_max(uint32_t v) {
#pragma unroll
    for (int o = 1; o < TEAM; o *= 2) v = max(v, (uint32_t)__shfl_xor((int)v, o, TEAM));
    return v;
}

__device__ __forceinline__ int64_t cache_row(const CacheParams &p, uint32_t slot, uint32_t head) {
    const uint32_t page = p.page.div(slot), off = slot - page * p.page.d;
    return ((int64_t)page * p.io.cache.heads + head) * p.page.d + off;
}

// T: type of the values given; C: the cache's (int8_t, or a value type).  A team takes a
// row of the keys and the same of the values, so that two loads are on their way at once and
// the slot is looked up once (32768 tokens x 8 heads x 128, bf16 to 8 bits: 61.6 us with a row
// to a team, 51.6 us, 3.9 TB/s, with both; two or four rows of each are slower again).
template <typename T, typename C, int TEAM>
__global__ __launch_bounds__(kThreads) void cache_write(const CacheParams p) {
    const uint32_t row = blockIdx.x * (kThreads / TEAM) + threadIdx.x / TEAM;
    const int d = (int)(threadIdx.x % TEAM) * 8, dim = p.io.cache.dim;
    if (row >= p.rows) return;
    const uint32_t token = p.heads.div(row), head = row - token * p.heads.d;
    const uint32_t slot = (uint32_t)p.io.slots[token];
    if (slot >= p.slots) return;  // negative slots are large numbers here
    const bool mine = d < dim;
    f32x8 x[2] = {};
    if (mine) {
        x[0] = Value<T>::load8((const T *)p.io.k + token * p.io.k_token + head * p.io.k_head + d);
        x[1] = Value<T>::load8((const T *)p.io.v + token * p.io.v_token + head * p.io.v_head + d);
    }
    const int64_t at = cache_row(p, slot, head);
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        C *dst = (C *)(side ? p.io.cache.v : p.io.cache.k) + at * dim + d;
        if constexpr (std::is_same_v<C, int8_t>) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, magnitude(x[side][i]));
            m = team_max<TEAM>(m);
            const float s = row_scale(m), inv = row_inverse(s, m);
            int c[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (inv != 0.f) row_codes8(x[side], s, inv, c);
            if (mine) *(u32x2 *)dst = u32x2{pack_codes(c[0], c[1], c[2], c[3]), pack_codes(c[4], c[5], c[6], c[7])};
            if (d == 0) (side ? p.io.cache.v_scale : p.io.cache.k_scale)[at] = s;
        } else {
            if (mine) Value<C>::store8(dst, x[side]);
        }
    }
}

// blockIdx.y: 0 keys, 1 values.
template <typename T, typename C, int TEAM>
__global__ __launch_bounds__(kThreads) void cache_read(const CacheParams p) {
    const uint32_t row = blockIdx.x * (kThreads / TEAM) + threadIdx.x / TEAM;
    const int d = (int)(threadIdx.x % TEAM) * 8, dim = p.io.cache.dim;
    const bool second = blockIdx.y != 0;
    if (row >= p.rows || d >= dim) return;
    const uint32_t token = p.heads.div(row), head = row - token * p.heads.d;
    const uint32_t slot = (uint32_t)p.io.slots[token];
    f32x8 x = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (slot < p.slots) {
        const int64_t at = cache_row(p, slot, head);
        const C *src = (const C *)(second ? p.io.cache.v : p.io.cache.k) + at * dim + d;
        if constexpr (std::is_same_v<C, int8_t>) {
            const u32x2 c = *(const u32x2 *)src;
            const float s = (second ? p.io.cache.v_scale : p.io.cache.k_scale)[at];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = (float)(int8_t)(c[i / 4] >> (8 * (i % 4))) * s;
        } else {
            x = Value<C>::load8(src);
        }
    }
    Value<T>::store8((T *)(second ? p.io.v_out : p.io.k_out) + (int64_t)row * dim + d, x);
}

template <typename T, typename C, int TEAM> hipError_t launch3(const CacheIo &a, bool write, hipStream_t st) {
    // one launch but for the largest calls: a launch holds fewer than 2^32 threads
    const int64_t heads = a.cache.heads, most = std::max<int64_t>(1, (1 << 26) / heads);
    hipError_t e = hipSuccess;
    for (int64_t t = 0; t < a.tokens && e == hipSuccess; t += most) {
        CacheParams p{a, make_fastdiv((uint32_t)heads), make_fastdiv((uint32_t)a.cache.page_size), 0,
                      (uint32_t)(a.cache.pages * a.cache.page_size)};
        p.rows = (uint32_t)(std::min(most, a.tokens - t) * heads);
        p.io.slots += t;
        const unsigned grid = (p.rows + kThreads / TEAM - 1) / (kThreads / TEAM);
        if (write) {
            p.io.k = (const T *)a.k + t * a.k_token;
            p.io.v = (const T *)a.v + t * a.v_token;
            cache_write<T, C, TEAM><<<grid, kThreads, 0, st>>>(p);
        } else {
            p.io.k_out = (T *)a.k_out + t * heads * a.cache.dim;
            p.io.v_out = (T *)a.v_out + t * heads * a.cache.dim;
            cache_read<T, C, TEAM><<<dim3(grid, 2), kThreads, 0, st>>>(p);
        }
        e = hipGetLastError();
    }
    return e;
}
template <typename T, typename C> hipError_t launch2(const CacheIo &a, bool write, hipStream_t st) {
    return a.cache.dim <= 128 ? launch3<T, C, 16>(a, write, st) : launch3<T, C, 32>(a, write, st);
}
template <typename T> hipError_t launch1(const CacheIo &a, bool write, hipStream_t st) {
    switch (a.cache.dtype) {
        case CBS_DTYPE_I8: return launch2<T, int8_t>(a, write, st);
        case CBS_DTYPE_F32: return launch2<T, float>(a, write, st);
        case CBS_DTYPE_BF16: return launch2<T, __bf16>(a, write, st);
        default: return launch2<T, _Float16>(a, write, st);
    }
}
hipError_t launch(const CacheIo &a, bool write, hipStream_t st) {
    switch (a.dtype) {
        case CBS_DTYPE_F32: return launch1<float>(a, write, st);
        case CBS_DTYPE_BF16: return launch1<__bf16>(a, write, st);
        default: return launch1<_Float16>(a, write, st);
    }
}

}  // namespace

hipError_t launch_cache_write(const CacheIo &a, hipStream_t st) { return launch(a, true, st); }
hipError_t launch_cache_read(const CacheIo &a, hipStream_t st) { return launch(a, false, st); }

}  // namespace cbs
