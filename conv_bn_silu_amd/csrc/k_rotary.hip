// k_rotary.hip -- rotary positions: the pairs of a head turned by position * frequency, of a
// tensor, or of queries and keys on their way out and into the paged cache, with the values.
//
// Angles.  position * frequency / 2 pi in turns, in 64 bits (fp32 would be off by 2^-25 of the
// position: 0.04 radians at a million); less the nearest quarter it fits fp32, where the series
// of sine and cosine on an eighth of a turn either way end below half a step.  A workgroup has a few tokens,
// works their angles out once, into LDS, and turns all their heads by them.
//
// Bound by HBM: every row is read once and written once.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "b8_device.h"
#include "st_launch.h"

namespace cbs {
namespace {

constexpr int kMostDim = 512, kMostPairs = kMostDim / 2;
constexpr int kMostThreads = 1024;

struct RotaryParams {
    RotaryArgs a;
    FastDiv rows;     // of a token: its queries, keys and values
    FastDiv page;
    uint32_t slots;   // pages * page size
    int64_t token, end;  // tokens of the launch
    int tokens;          // to a workgroup
};

// (cos, sin) of position * frequency, times the magnitude.
__device__ __forceinline__ float2 turn_of(const cbs_rotary &r, int position, int pair) {
    constexpr double kTurns = 0.15915494309189533577;  // 1 / 2 pi
    const double t = (double)position * r.frequencies[pair] * kTurns;
    const double quarter = __builtin_rint(4 * t);
    const float x = (float)__builtin_fma(-0.25, quarter, t) * 6.28318530717958648f;  // within pi / 4
    const int q = (int)(quarter - 4 * __builtin_floor(quarter * 0.25));
    const float z = x * x;
    // Taylor's; the terms left out are below 2^-29 of one
    const float s = x + x * z * (-1.f / 6 + z * (1.f / 120 + z * (-1.f / 5040 + z * (1.f / 362880))));
    const float c = 1.f + z * (-0.5f + z * (1.f / 24 + z * (-1.f / 720 + z * (1.f / 40320 + z * (-1.f / 3628800)))));
    const float cos = q == 0 ? c : q == 1 ? -s : q == 2 ? -c : s, sin = q == 0 ? s : q == 1 ? c : q == 2 ? -s : -c;
    return {cos * r.magnitude, sin * r.magnitude};
}
__device__ __forceinline__ void turn(float &a, float &b, float2 by) {
    const float x = a;
    a = x * by.x - b * by.y;
    b = b * by.x + x * by.y;
}

// A row of a token: its tensor, and where it goes.
template <typename T> struct Row {
    const T *from;
    T *to;               // queries
    int side;            // 0 queries, 1 keys, 2 values
    int64_t at;          // keys and values: their row of the cache, -1 for nowhere
    __device__ __forceinline__ Row(const RotaryParams &p, int64_t token, int row) {
        const RotaryArgs &a = p.a;
        side = row < a.heads ? 0 : row < a.heads + a.kv_heads ? 1 : 2;
        to = nullptr, at = -1;
        if (side == 0) {
            from = (const T *)a.q + token * a.q_token + row * a.q_head;
            to = (T *)a.q_out + token * a.out_token + row * a.out_head;
            return;
        }
        const int head = row - a.heads - (side == 2 ? a.kv_heads : 0);
        from = side == 1 ? (const T *)a.k + token * a.k_token + head * a.k_head : (const T *)a.v + token * a.v_token + head * a.v_head;
        const uint32_t slot = (uint32_t)a.slots[token];
        if (slot < p.slots) {  // negative slots are large numbers here
            const uint32_t page = p.page.div(slot);
            at = ((int64_t)page * a.cache.heads + head) * p.page.d + (slot - page * p.page.d);
        }
    }
};

// A workgroup's angles, by all of its threads.
__device__ __forceinline__ void fill_turns(const RotaryParams &p, float2 *turns, int64_t token0, int tokens) {
    const int pairs = p.a.rotary.pairs;
    for (int i = (int)threadIdx.x; i < tokens * pairs; i += (int)blockDim.x) {
        const int t = i / pairs;
        turns[i] = turn_of(p.a.rotary, p.a.positions[token0 + t], i - t * pairs);
    }
    __syncthreads();
}

// Where dims and pairs come in whole 8s: a row belongs to a team of LANES lanes, two pieces of 8 a lane,
// of which a lane of the turned part has both halves of its pairs.  C: the cache's type (without a cache,
// T).
template <typename T, typename C, int LANES, bool INTERLEAVED>
__global__ __launch_bounds__(kMostThreads) void rotary_pieces(const RotaryParams p) {
    extern __shared__ float2 turns[];
    const RotaryArgs &a = p.a;
    const int64_t token0 = p.token + (int64_t)blockIdx.x * p.tokens;
    const int tokens = (int)min((int64_t)p.tokens, p.end - token0);
    fill_turns(p, turns, token0, tokens);

    const int lane = (int)threadIdx.x % LANES, pairs = a.rotary.pairs, half = pairs / 8;
    // the lane's pieces, and whether they are turned; past dim there is nothing
    const bool turned = INTERLEAVED ? 16 * lane < 2 * pairs : lane < half;
    const int d0 = INTERLEAVED || lane >= half ? 16 * lane : 8 * lane, d1 = INTERLEAVED || lane >= half ? d0 + 8 : d0 + pairs;
    const bool has0 = d0 < a.dim, has1 = d1 < a.dim;
    const int team = (int)threadIdx.x / LANES, teams = (int)blockDim.x / LANES;
    for (int i = team; i < tokens * (int)p.rows.d; i += teams) {
        const int t = (int)p.rows.div((uint32_t)i);
        const Row<T> row(p, token0 + t, i - t * (int)p.rows.d);
        if (row.side != 0 && row.at < 0) continue;
        f32x8 x[2] = {};
        if (has0) x[0] = Value<T>::load8(row.from + d0);
        if (has1) x[1] = Value<T>::load8(row.from + d1);
        if (turned && row.side != 2) {
            const float2 *by = turns + t * pairs;
            if constexpr (INTERLEAVED) {
#pragma unroll
                for (int side = 0; side < 2; ++side)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int pair = 8 * lane + 4 * side + e;
                        if (pair < pairs) {
                            float u = x[side][2 * e], v = x[side][2 * e + 1];
                            turn(u, v, by[pair]);
                            x[side][2 * e] = u, x[side][2 * e + 1] = v;
                        }
                    }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float u = x[0][e], v = x[1][e];
                    turn(u, v, by[8 * lane + e]);
                    x[0][e] = u, x[1][e] = v;
                }
            }
        }
        if (row.side == 0) {
            if (has0) Value<T>::store8(row.to + d0, x[0]);
            if (has1) Value<T>::store8(row.to + d1, x[1]);
            continue;
        }
        C *const to = (C *)(row.side == 1 ? a.cache.k : a.cache.v) + row.at * a.dim;
        if constexpr (std::is_same_v<C, int8_t>) {
            uint32_t top = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) top = max(top, max(magnitude(x[0][e]), magnitude(x[1][e])));
#pragma unroll
            for (int o = 1; o < LANES; o *= 2) top = max(top, (uint32_t)__shfl_xor((int)top, o, LANES));
            const float s = row_scale(top), inv = row_inverse(s, top);
#pragma unroll
            for (int side = 0; side < 2; ++side) {
                int c[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                if (inv != 0.f) row_codes8(x[side], s, inv, c);
                if (side ? has1 : has0)
                    *(u32x2 *)(to + (side ? d1 : d0)) = u32x2{pack_codes(c[0], c[1], c[2], c[3]), pack_codes(c[4], c[5], c[6], c[7])};
            }
            if (lane == 0) (row.side == 1 ? a.cache.k_scale : a.cache.v_scale)[row.at] = s;
        } else {
            if (has0) Value<C>::store8(to + d0, x[0]);
            if (has1) Value<C>::store8(to + d1, x[1]);
        }
    }
}

// Any dims and pairs: a wave to a row, every 64th value a lane.  A row goes through LDS, where each
// value finds its partner.  All of a row is read before any of it is written, which may be in its place.
template <typename T, typename C>
__global__ __launch_bounds__(256) void rotary_values(const RotaryParams p) {
    constexpr int kEach = kMostDim / 64;
    __shared__ float2 turns[kMostPairs];
    __shared__ float rows[4][kMostDim];
    const RotaryArgs &a = p.a;
    const int64_t token = p.token + (int64_t)blockIdx.x;
    fill_turns(p, turns, token, 1);
    const int lane = (int)threadIdx.x % 64, wave = (int)threadIdx.x / 64, pairs = a.rotary.pairs;
    float *const mine = rows[wave];
    for (int r = wave; r < (int)p.rows.d; r += 4) {
        const Row<T> row(p, token, r);
        if (row.side != 0 && row.at < 0) continue;
        float x[kEach];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int d = lane + 64 * i;
            x[i] = d < a.dim ? Value<T>::load1(row.from + d) : 0.f;
            mine[d] = x[i];
        }
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int d = lane + 64 * i;
            if (row.side != 2 && d < 2 * pairs) {
                const bool second = a.rotary.interleaved ? d % 2 != 0 : d >= pairs;
                const int pair = a.rotary.interleaved ? d / 2 : second ? d - pairs : d;
                const float other = mine[a.rotary.interleaved ? d ^ 1 : second ? pair : d + pairs];
                float u = second ? other : x[i], v = second ? x[i] : other;
                turn(u, v, turns[pair]);
                x[i] = second ? v : u;
            }
            top = max(top, magnitude(x[i]));
        }
        __builtin_amdgcn_wave_barrier();
        if (row.side == 0) {
#pragma unroll
            for (int i = 0; i < kEach; ++i)
                if (lane + 64 * i < a.dim) Value<T>::store1(row.to + lane + 64 * i, x[i]);
            continue;
        }
        C *const to = (C *)(row.side == 1 ? a.cache.k : a.cache.v) + row.at * a.dim;
        if constexpr (std::is_same_v<C, int8_t>) {
#pragma unroll
            for (int o = 1; o < 64; o *= 2) top = max(top, (uint32_t)__shfl_xor((int)top, o, 64));
            const float s = row_scale(top), inv = row_inverse(s, top);
            const f32x8 all = {x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7]};
            int c[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (inv != 0.f) row_codes8(all, s, inv, c);
#pragma unroll
            for (int i = 0; i < kEach; ++i)
                if (lane + 64 * i < a.dim) to[lane + 64 * i] = (int8_t)c[i];
            if (lane == 0) (row.side == 1 ? a.cache.k_scale : a.cache.v_scale)[row.at] = s;
        } else {
#pragma unroll
            for (int i = 0; i < kEach; ++i)
                if (lane + 64 * i < a.dim) Value<C>::store1(to + lane + 64 * i, x[i]);
        }
    }
}

template <typename T, typename C, int LANES, bool INTERLEAVED> void launch_pieces(const RotaryParams &p, int64_t tokens, hipStream_t st) {
    RotaryParams q = p;
    const int64_t each = (int64_t)p.rows.d * LANES;  // threads to a token
    q.tokens = (int)std::max<int64_t>(1, std::min<int64_t>(256 / each, 8));
    const int threads = (int)std::min<int64_t>(kMostThreads, (q.tokens * each + 63) / 64 * 64);
    rotary_pieces<T, C, LANES, INTERLEAVED><<<(unsigned)((tokens + q.tokens - 1) / q.tokens), threads,
                                              q.tokens * p.a.rotary.pairs * sizeof(float2), st>>>(q);
}
template <typename T, typename C, int LANES> void launch_lanes(const RotaryParams &p, int64_t tokens, hipStream_t st) {
    if (p.a.rotary.interleaved) launch_pieces<T, C, LANES, true>(p, tokens, st);
    else launch_pieces<T, C, LANES, false>(p, tokens, st);
}

template <typename T, typename C> hipError_t launch2(const RotaryArgs &a, hipStream_t st) {
    const int rows = a.heads + 2 * a.kv_heads;
    RotaryParams p{a, make_fastdiv((uint32_t)rows), make_fastdiv((uint32_t)std::max(1, a.cache.page_size)),
                   (uint32_t)(a.kv_heads ? a.cache.pages * a.cache.page_size : 0), 0, 0, 1};
    const bool pieces = a.dim % 8 == 0 && (a.rotary.interleaved || a.rotary.pairs % 8 == 0);
    // one launch but for the largest calls: a launch holds fewer than 2^32 threads
    constexpr int64_t kMost = 1 << 21;
    for (; p.token < a.tokens; p.token += kMost) {
        const int64_t tokens = std::min(kMost, a.tokens - p.token);
        p.end = p.token + tokens;
        if (!pieces) rotary_values<T, C><<<(unsigned)tokens, 256, 0, st>>>(p);
        else if (a.dim <= 128) launch_lanes<T, C, 8>(p, tokens, st);
        else if (a.dim <= 256) launch_lanes<T, C, 16>(p, tokens, st);
        else if constexpr (std::is_same_v<T, C>) launch_lanes<T, C, 32>(p, tokens, st);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}
template <typename T> hipError_t launch1(const RotaryArgs &a, hipStream_t st) {
    if (a.kv_heads == 0) return launch2<T, T>(a, st);
    switch (a.cache.dtype) {
        case CBS_DTYPE_I8: return launch2<T, int8_t>(a, st);
        case CBS_DTYPE_F32: return launch2<T, float>(a, st);
        case CBS_DTYPE_BF16: return launch2<T, __bf16>(a, st);
        default: return launch2<T, _Float16>(a, st);
    }
}

}  // namespace

hipError_t launch_rotary(const RotaryArgs &a, hipStream_t st) {
    switch (a.dtype) {
        case CBS_DTYPE_F32: return launch1<float>(a, st);
        case CBS_DTYPE_BF16: return launch1<__bf16>(a, st);
        default: return launch1<_Float16>(a, st);
    }
}

}  // namespace cbs
