// k_rotary.hip -- rotary positions: the pairs of a head turned by position * frequency, of a
// tensor, or of queries and keys on their way out and into the paged cache, with the values.
//
// Angles.  position * frequency / 2 pi in turns, in 64 bits (fp32 would be off by 2^-25 of the
// position: 0.04 radians at a million); less the nearest quarter it fits fp32, where the series
// of sine and cosine on an eighth of a turn either way end below half a step.  A workgroup works its tokens'
// angles out once, into LDS, while its first rows are on their way.
//
// Bound by HBM: every row is read once and written once.  32768 tokens, 32 heads over 8, dim 128, bf16 into
// 8 bits: 128 us, 5.8 TB/s (741 MB; a large copy: 6.3 TB/s, 118 us).  Queries, keys and values go to different
// workgroups, whose addresses and branches are then the same for all lanes (a workgroup with all rows of
// a token, each lane looking up its own: 185 us, 250 vector instructions a row of 16 lanes' values); a team takes two rows at
// most, one after the other (eight: 146).  Other forms of 32768 tokens, us and what a copy would take: into 16 bits 150, 128;
// fp32 into 8 bits 271, 224; into 8 bits 64 heads over 8 of dim 64 134, 102, 16 over 4 of dim 256 130, 117, 8 over 8 of dim 128
// 62, 54.  8192 tokens 33, 29, of 40 heads without a cache 29, 27; 5001 ragged ones (15 over 5, dim 80, fp16) 10, 6; 64 tokens
// 4.7 on the GPU, 8 a call.  Pairs that are no whole 8s make smaller pieces: 24 heads over 8 of dim 80, 20 pairs, into 8
// bits 134, 60; 32 of dim 100, 50 pairs, without a cache 99, 67 (odd numbers of pairs, through LDS: 25 197, 49 168).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "b8_device.h"
#include "st_device.h"
#include "st_launch.h"

namespace cbs {
namespace {


struct RotaryParams {
    RotaryArgs a;
    FastDiv page;
    uint32_t slots;   // pages * page size
    int64_t token, end;  // tokens of the launch
    // workgroups of the queries and of the keys (and of the values), tokens of each; the keys, whose workgroups take
    // longest, go first (8192 tokens 43 -> 39 us)
    int q_blocks, kv_blocks, q_tokens, kv_tokens;
    FastDiv q_heads, kv_heads, pairs;
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

__device__ __forceinline__ int64_t cache_line(const RotaryParams &p, uint32_t slot, int head) {
    const uint32_t page = p.page.div(slot);
    return ((int64_t)page * p.a.cache.heads + head) * p.page.d + (slot - page * p.page.d);
}

constexpr int kMostThreads = 512;

// P values as T holds them, at any address.
template <typename T, int P> struct Piece {
    static constexpr int kWords = P * (int)sizeof(T) / 4, kParts = kWords > 4 ? kWords / 4 : 1;
    typedef uint32_t words __attribute__((ext_vector_type(kWords / kParts)));
    typedef T values __attribute__((ext_vector_type(P)));
    typedef float floats __attribute__((ext_vector_type(P)));
    typedef words __attribute__((aligned(1))) any;
    struct Raw {
        words w[kParts];
    } raw;
    Piece() = default;
    __device__ __forceinline__ explicit Piece(const float *x) {
        floats v;
#pragma unroll
        for (int e = 0; e < P; ++e) v[e] = x[e];
        raw = __builtin_bit_cast(Raw, __builtin_convertvector(v, values));
    }
    template <bool STREAM> __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int i = 0; i < kParts; ++i) raw.w[i] = STREAM ? __builtin_nontemporal_load((const any *)p + i) : ((const any *)p)[i];
    }
    template <bool STREAM> __device__ __forceinline__ void store(T *p) const {
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            if constexpr (STREAM) __builtin_nontemporal_store(raw.w[i], (any *)p + i);
            else ((any *)p)[i] = raw.w[i];
        }
    }
    __device__ __forceinline__ void get(float *x) const {
        const floats v = __builtin_convertvector(__builtin_bit_cast(values, raw), floats);
#pragma unroll
        for (int e = 0; e < P; ++e) x[e] = v[e];
    }
};

// Where the angle of pair i of a token lies in LDS: lanes read P of them, two at a time, and so side by side.
template <int P> __device__ __forceinline__ int turn_at(int i, int pairs) { return i % P / 2 * (pairs / P * 2) + i / P * 2 + i % 2; }

// Where dims and pairs come in whole Ps (8, 4 or 2): a row belongs to a team of LANES lanes, two pieces of P a
// lane, of which a lane of the turned part has both halves of its pairs.  A workgroup has the queries, the keys or
// the values (SIDE) of some tokens, and while a team turns one row the next one is on its way.  C: the
// cache's type (without a cache, T).  STREAM: the tensors pass by the caches.
template <typename T, typename C, int P, int LANES, bool INTERLEAVED, bool STREAM, int SIDE>
__device__ __forceinline__ void rotary_side(const RotaryParams &p, int block, float2 *turns) {
    const RotaryArgs &a = p.a;
    const int teams = (int)blockDim.x / LANES;
    const int each = SIDE == 0 ? p.q_tokens : p.kv_tokens, heads = SIDE == 0 ? a.heads : a.kv_heads;
    const int64_t token0 = p.token + (int64_t)block * each;
    const int tokens = (int)min((int64_t)each, p.end - token0), tasks = tokens * heads;
    const FastDiv &by_heads = SIDE == 0 ? p.q_heads : p.kv_heads;
    const int64_t token_step = SIDE == 0 ? a.q_token : SIDE == 1 ? a.k_token : a.v_token;
    const int64_t head_step = SIDE == 0 ? a.q_head : SIDE == 1 ? a.k_head : a.v_head;
    const T *const from = (const T *)(SIDE == 0 ? a.q : SIDE == 1 ? a.k : a.v) + token0 * token_step;

    const int lane = (int)threadIdx.x % LANES, pairs = a.rotary.pairs, half = pairs / P, team = (int)threadIdx.x / LANES;
    // the lane's pieces, and whether they are turned; past dim there is nothing
    const bool turned = INTERLEAVED ? P * lane < pairs : lane < half;
    const bool apart = !INTERLEAVED && lane < half;  // the second is not the one after the first
    const int d0 = apart ? P * lane : 2 * P * lane, d1 = apart ? d0 + pairs : d0 + P;
    const bool has0 = d0 < a.dim, has1 = d1 < a.dim;
    // the lane's angles: two side by side, the next two `stride` further
    const bool whole = !INTERLEAVED || pairs % P == 0;
    const int first = whole ? 2 * lane : P * lane, stride = whole ? pairs / P * 2 : 2;

    Piece<T, P> next[2] = {};
    uint32_t next_slot = 0;
    auto take = [&](int i) {
        const int t = (int)by_heads.div((uint32_t)i), h = i - t * heads;
        const T *const row = from + t * token_step + h * head_step;
        if (has0) next[0].template load<STREAM>(row + d0);
        if (has1) next[1].template load<STREAM>(row + d1);
        if constexpr (SIDE != 0) next_slot = (uint32_t)a.slots[token0 + t];
    };
    if (team < tasks) take(team);
    if constexpr (SIDE != 2) {
        for (int i = (int)threadIdx.x; i < tokens * pairs; i += (int)blockDim.x) {
            const int t = (int)p.pairs.div((uint32_t)i), pair = i - t * pairs;
            turns[t * pairs + (whole ? turn_at<P>(pair, pairs) : pair)] = turn_of(a.rotary, a.positions[token0 + t], pair);
        }
        __syncthreads();
    }
    for (int i = team; i < tasks; i += teams) {
        float x[2 * P];
        next[0].get(x), next[1].get(x + P);
        const uint32_t slot = next_slot;
        if (i + teams < tasks) take(i + teams);
        const int t = (int)by_heads.div((uint32_t)i), h = i - t * heads;
        if (SIDE != 2 && turned) {
            const float2 *const by = turns + t * pairs + first;
            if (whole) {
#pragma unroll
                for (int e = 0; e < P; ++e) turn(x[INTERLEAVED ? 2 * e : e], x[INTERLEAVED ? 2 * e + 1 : P + e], by[e / 2 * stride + e % 2]);
            } else {
#pragma unroll
                for (int e = 0; e < P; ++e)
                    if (P * lane + e < pairs) turn(x[2 * e], x[2 * e + 1], by[e]);
            }
        }
        if constexpr (SIDE == 0) {
            T *const to = (T *)a.q_out + token0 * a.out_token + t * a.out_token + h * a.out_head;
            if (has0) Piece<T, P>(x).template store<STREAM>(to + d0);
            if (has1) Piece<T, P>(x + P).template store<STREAM>(to + d1);
        } else {
            if (slot >= p.slots) continue;  // negative slots are large numbers here
            const int64_t line = cache_line(p, slot, h);
            C *const to = (C *)(SIDE == 1 ? a.cache.k : a.cache.v) + line * a.dim;
            if constexpr (std::is_same_v<C, int8_t>) {
                uint32_t top = 0;
#pragma unroll
                for (int e = 0; e < 2 * P; ++e) top = max(top, magnitude(x[e]));
                top = team_max_of<LANES>(top);
                const float s = row_scale(top), inv = row_quotient(s, top);
                u32x2 codes[2] = {};
#pragma unroll
                for (int g = 0; g < (2 * P + 7) / 8; ++g) {
                    f32x8 v = {};
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (8 * g + e < 2 * P) v[e] = x[8 * g + e];
                    if (inv != 0.f) codes[g] = codes_of8(v, s, inv);
                }
                if constexpr (P == 8) {
                    // pieces that lie apart: two lanes exchange one each, for stores of 16 bytes
                    const bool odd = lane & 1, trade = !INTERLEAVED && lane < (half & ~1);
                    const u32x2 give = odd ? codes[0] : codes[1];
                    const u32x2 got = {lane_from<kSwap1>(give.x, give.x), lane_from<kSwap1>(give.y, give.y)};
                    if (trade || (!apart && has1)) {
                        const u32x2 lo = trade && odd ? got : codes[0], hi = trade && !odd ? got : codes[1];
                        ((Any16 *)(to + (trade && odd ? d1 - 8 : d0)))->v = u32x4{lo.x, lo.y, hi.x, hi.y};
                    } else {
                        if (has0) *(u32x2 *)(to + d0) = codes[0];
                        if (has1) *(u32x2 *)(to + d1) = codes[1];
                    }
                } else {
                    if constexpr (P == 4) {
                        if (has0) *(uint32_t *)(to + d0) = codes[0].x;
                        if (has1) *(uint32_t *)(to + d1) = codes[0].y;
                    } else {
                        if (has0) *(uint16_t *)(to + d0) = (uint16_t)codes[0].x;
                        if (has1) *(uint16_t *)(to + d1) = (uint16_t)(codes[0].x >> 16);
                    }
                }
                if (lane == 0) (SIDE == 1 ? a.cache.k_scale : a.cache.v_scale)[line] = s;
            } else {
                if (has0) Piece<C, P>(x).template store<false>(to + d0);
                if (has1) Piece<C, P>(x + P).template store<false>(to + d1);
            }
        }
    }
}

template <typename T, typename C, int P, int LANES, bool INTERLEAVED, bool STREAM>
__global__ __launch_bounds__(kMostThreads) void rotary_pieces(const RotaryParams p) {
    extern __shared__ __attribute__((aligned(16))) float2 turns[];
    const int block = (int)blockIdx.x;
    if (block < p.kv_blocks) rotary_side<T, C, P, LANES, INTERLEAVED, STREAM, 1>(p, block, turns);
    else if (block < 2 * p.kv_blocks) rotary_side<T, C, P, LANES, INTERLEAVED, STREAM, 2>(p, block - p.kv_blocks, turns);
    else rotary_side<T, C, P, LANES, INTERLEAVED, STREAM, 0>(p, block - 2 * p.kv_blocks, turns);
}

// Any dims and pairs: 8 dims a lane, each of which finds its partner in LDS, where the row lies in fp32; the last
// lane of a row may have fewer.  All of a row is read before any of it is written, which may be in its place.
template <typename T, typename C, int LANES, int SIDE>
__device__ __forceinline__ void rotary_side_any(const RotaryParams &p, int block, float *rows, float2 *turns) {
    const RotaryArgs &a = p.a;
    const int teams = (int)blockDim.x / LANES;
    const int each = SIDE == 0 ? p.q_tokens : p.kv_tokens, heads = SIDE == 0 ? a.heads : a.kv_heads;
    const int64_t token0 = p.token + (int64_t)block * each;
    const int tokens = (int)min((int64_t)each, p.end - token0), tasks = tokens * heads;
    const FastDiv &by_heads = SIDE == 0 ? p.q_heads : p.kv_heads;
    const int64_t token_step = SIDE == 0 ? a.q_token : SIDE == 1 ? a.k_token : a.v_token;
    const int64_t head_step = SIDE == 0 ? a.q_head : SIDE == 1 ? a.k_head : a.v_head;
    const T *const from = (const T *)(SIDE == 0 ? a.q : SIDE == 1 ? a.k : a.v) + token0 * token_step;
    const int lane = (int)threadIdx.x % LANES, pairs = a.rotary.pairs, team = (int)threadIdx.x / LANES, d = 8 * lane;
    float *const mine = rows + team * LANES * 8;

    Held<T> next = {};
    uint32_t next_slot = 0;
    auto take = [&](int i) {
        const int t = (int)by_heads.div((uint32_t)i), h = i - t * heads;
        next = Held<T>(load_chunk(from + t * token_step + h * head_step, d, a.dim));
        if constexpr (SIDE != 0) next_slot = (uint32_t)a.slots[token0 + t];
    };
    if (team < tasks) take(team);
    if constexpr (SIDE != 2) {
        for (int i = (int)threadIdx.x; i < tokens * pairs; i += (int)blockDim.x) {
            const int t = (int)p.pairs.div((uint32_t)i);
            turns[i] = turn_of(a.rotary, a.positions[token0 + t], i - t * pairs);
        }
        __syncthreads();
    }
    for (int i = team; i < tasks; i += teams) {
        f32x8 x = next.get();
        const uint32_t slot = next_slot;
        if (i + teams < tasks) take(i + teams);
        const int t = (int)by_heads.div((uint32_t)i), h = i - t * heads;
        if constexpr (SIDE != 2) {
            const float2 *const by = turns + t * pairs;
            if (a.rotary.interleaved) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (d / 2 + e < pairs) {
                        float u = x[2 * e], v = x[2 * e + 1];
                        turn(u, v, by[d / 2 + e]);
                        x[2 * e] = u, x[2 * e + 1] = v;
                    }
            } else {
                *(f32x4 *)(mine + d) = f32x4{x[0], x[1], x[2], x[3]};
                *(f32x4 *)(mine + d + 4) = f32x4{x[4], x[5], x[6], x[7]};
                __builtin_amdgcn_wave_barrier();
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int at = d + e;
                    if (at >= 2 * pairs) continue;
                    const bool second = at >= pairs;
                    const float other = mine[second ? at - pairs : at + pairs];
                    float u = second ? other : x[e], v = second ? x[e] : other;
                    turn(u, v, by[second ? at - pairs : at]);
                    x[e] = second ? v : u;
                }
                __builtin_amdgcn_wave_barrier();
            }
        }
        if constexpr (SIDE == 0) {
            T *const to = (T *)a.q_out + token0 * a.out_token + t * a.out_token + h * a.out_head;
            if (d < a.dim) Held<T>(x).store_chunk(to, d, a.dim);
        } else {
            if (slot >= p.slots) continue;  // negative slots are large numbers here
            const int64_t line = cache_line(p, slot, h);
            C *const to = (C *)(SIDE == 1 ? a.cache.k : a.cache.v) + line * a.dim + d;
            if constexpr (std::is_same_v<C, int8_t>) {
                uint32_t top = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) top = max(top, magnitude(x[e]));
                top = team_max_of<LANES>(top);
                const float s = row_scale(top), inv = row_quotient(s, top);
                // a cache's rows are whole 8s
                if (d < a.dim) *(u32x2 *)to = inv != 0.f ? codes_of8(x, s, inv) : u32x2{0u, 0u};
                if (lane == 0) (SIDE == 1 ? a.cache.k_scale : a.cache.v_scale)[line] = s;
            } else {
                if (d < a.dim) Value<C>::store8(to, x);
            }
        }
    }
}

template <typename T, typename C, int LANES> __global__ __launch_bounds__(kMostThreads) void rotary_any(const RotaryParams p) {
    extern __shared__ __attribute__((aligned(16))) float2 turns[];
    __shared__ __attribute__((aligned(16))) float rows[kMostThreads * 8];
    const int block = (int)blockIdx.x;
    if (block < p.kv_blocks) rotary_side_any<T, C, LANES, 1>(p, block, rows, turns);
    else if (block < 2 * p.kv_blocks) rotary_side_any<T, C, LANES, 2>(p, block - p.kv_blocks, rows, turns);
    else rotary_side_any<T, C, LANES, 0>(p, block - 2 * p.kv_blocks, rows, turns);
}

// How a launch of teams of LANES lanes is divided.
struct Division {
    unsigned grid;
    int threads;
    size_t lds;
};
Division divide(RotaryParams &q, int64_t tokens, int lanes) {
    const RotaryArgs &a = q.a;
    q.q_heads = make_fastdiv((uint32_t)std::max(1, a.heads)), q.kv_heads = make_fastdiv((uint32_t)std::max(1, a.kv_heads));
    q.pairs = make_fastdiv((uint32_t)a.rotary.pairs);
    // A team takes two rows one after the other where that leaves enough workgroups.  The threads of a
    // workgroup: those that leave the fewest idle.
    const int64_t rows = a.heads + 2 * (int64_t)a.kv_heads, turns = tokens * rows * lanes > 2 * 256 * 2048 ? 2 : 1;
    const int64_t most = 4096 / a.rotary.pairs;  // tokens, by the angles' 32 KiB
    auto share = [&](int64_t heads, int64_t threads) {
        return (int)std::max<int64_t>(1, std::min<int64_t>(most, turns * threads / (heads * lanes)));
    };
    const int64_t first = std::max(1, a.heads ? a.heads : a.kv_heads);
    int threads = 0;
    double best = 0;
    for (int n : {256, 320, 384, 448, 512, 192}) {
        const int64_t busy_lanes = share(first, n) * first * lanes;
        const double busy = (double)busy_lanes / (double)((busy_lanes + n - 1) / n * n);
        if (busy > best + 0.02) best = busy, threads = n;
    }
    q.q_tokens = share(std::max(1, a.heads), threads), q.kv_tokens = share(std::max(1, a.kv_heads), threads);
    // The scales of a page's tokens lie side by side for a head: into 8 bits a workgroup has twice as many of them
    // where that leaves one for every second CU (2048 tokens, 32 heads over 8, 10.2 -> 9.6 us, 32768 129 -> 128, dim 80
    // with 20 pairs 141 -> 133; four times 11.9, 125 and 129; values of 32 bits 270 and 272).
    if (a.kv_heads && a.cache.dtype == CBS_DTYPE_I8 && a.dtype != CBS_DTYPE_F32 && tokens >= 256 * (int64_t)q.kv_tokens)
        q.kv_tokens = (int)std::min<int64_t>(most, 2 * q.kv_tokens);
    q.q_blocks = a.heads ? (int)((tokens + q.q_tokens - 1) / q.q_tokens) : 0;
    q.kv_blocks = a.kv_heads ? (int)((tokens + q.kv_tokens - 1) / q.kv_tokens) : 0;
    const int at_once = std::max(a.heads ? q.q_tokens : 0, a.kv_heads ? q.kv_tokens : 0);
    return Division{(unsigned)(q.q_blocks + 2 * q.kv_blocks), threads, at_once * a.rotary.pairs * sizeof(float2)};
}
template <typename T, typename C, int P, int LANES> void launch_pieces(RotaryParams p, int64_t tokens, hipStream_t st) {
    const Division d = divide(p, tokens, LANES);
    const int64_t bytes = tokens * (p.a.heads + 2 * (int64_t)p.a.kv_heads) * p.a.dim * 2 * (int64_t)sizeof(T);
    if constexpr (P == 8) {
        if (bytes > kCached) {
            if (p.a.rotary.interleaved) rotary_pieces<T, C, P, LANES, true, true><<<d.grid, d.threads, d.lds, st>>>(p);
            else rotary_pieces<T, C, P, LANES, false, true><<<d.grid, d.threads, d.lds, st>>>(p);
            return;
        }
    }
    if (p.a.rotary.interleaved) rotary_pieces<T, C, P, LANES, true, false><<<d.grid, d.threads, d.lds, st>>>(p);
    else rotary_pieces<T, C, P, LANES, false, false><<<d.grid, d.threads, d.lds, st>>>(p);
}
template <typename T, typename C, int LANES> void launch_any(RotaryParams p, int64_t tokens, hipStream_t st) {
    const Division d = divide(p, tokens, LANES);
    rotary_any<T, C, LANES><<<d.grid, d.threads, d.lds, st>>>(p);
}
// Caches have dims up to 256.
template <typename T, typename C, int P> void launch_by_dim(const RotaryParams &p, int64_t tokens, hipStream_t st) {
    if (p.a.dim <= 128) launch_pieces<T, C, P, 64 / P>(p, tokens, st);
    else if (p.a.dim <= 256) launch_pieces<T, C, P, 128 / P>(p, tokens, st);
    else if constexpr (std::is_same_v<T, C> && P > 2) launch_pieces<T, C, P, 256 / P>(p, tokens, st);
}

template <typename T, typename C> hipError_t launch2(const RotaryArgs &a, hipStream_t st) {
    RotaryParams p{a, make_fastdiv((uint32_t)std::max(1, a.cache.page_size)),
                   (uint32_t)(a.kv_heads ? a.cache.pages * a.cache.page_size : 0), 0, 0};
    // the largest pieces that dims and, of halves, pairs are whole numbers of
    auto whole = [&](int n) { return a.dim % n == 0 && (a.rotary.interleaved || a.rotary.pairs % n == 0); };
    const int piece = whole(8) ? 8 : whole(4) ? 4 : whole(2) && a.dim <= 256 ? 2 : 1;
    // one launch but for the largest calls: a launch holds fewer than 2^32 threads
    constexpr int64_t kMost = 1 << 21;
    for (; p.token < a.tokens; p.token += kMost) {
        const int64_t tokens = std::min(kMost, a.tokens - p.token);
        p.end = p.token + tokens;
        if (piece == 8) launch_by_dim<T, C, 8>(p, tokens, st);
        else if (piece == 4) launch_by_dim<T, C, 4>(p, tokens, st);
        else if (piece == 2) launch_by_dim<T, C, 2>(p, tokens, st);
        else if (a.dim <= 128) launch_any<T, C, 16>(p, tokens, st);
        else if (a.dim <= 256) launch_any<T, C, 32>(p, tokens, st);
        else if constexpr (std::is_same_v<T, C>) launch_any<T, C, 64>(p, tokens, st);
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
