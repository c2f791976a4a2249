// k_norm.hip -- the residual's addition with the root-mean-square norm:
// h = x + residual, y = h w / sqrt(mean(h^2) + eps), y in x's type or as rows in 8 bits.
//
// Bound by HBM: x and the residual are read once, h and y written once.  A row belongs to a
// team of lanes and stays in their registers, 32 values a lane, from the sum of its squares to
// y; longer rows read h a second time.
//
// Squares are summed in 64 bits: no row of finite numbers overflows or vanishes on the way, and
// the matter is hidden under the loads (a CU has some 200 cycles for 64 values there).  r = 1 /
// sqrt(...) and h r are in 64 bits too: where h is large, r lies below fp32's normal numbers.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "b8_device.h"
#include "b8_linear.h"
#include "st_launch.h"

namespace cbs {
namespace {

constexpr int kChunks = 4;  // of 8 values a lane keeps

// 8 values from k on, zeros from K on.
template <typename T> __device__ __forceinline__ f32x8 load_chunk(const T *row, int k, int K) {
    f32x8 x = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (k + 8 <= K) return Value<T>::load8(row + k);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (k + i < K) x[i] = Value<T>::load1(row + k + i);
    return x;
}
template <typename T> __device__ __forceinline__ void store_chunk(T *row, int k, int K, f32x8 v) {
    if (k + 8 <= K) {
        Value<T>::store8(row + k, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (k + i < K) Value<T>::store1(row + k + i, v[i]);
}

struct NormParams {
    NormArgs a;
    CodesLayout l;  // of y in 8 bits
    int m0;         // row that the launch begins with
};

// T: type of x and y, R: of the residual and the sum.  TEAM lanes to a row, 64 or more of them a
// workgroup of their own waves.
template <typename T, typename R, int TEAM, bool INT8>
__global__ __launch_bounds__(TEAM < 256 ? 256 : TEAM) void add_rms_norm(const NormParams p) {
    constexpr int kThreads = TEAM < 256 ? 256 : TEAM, kWaves = TEAM / 64;
    __shared__ double squares_of[kWaves > 0 ? kWaves : 1];
    __shared__ uint32_t top_of[kWaves > 0 ? kWaves : 1];
    const NormArgs &a = p.a;
    const int lane = (int)threadIdx.x % TEAM, K = a.K;
    const int m = p.m0 + (int)blockIdx.x * (kThreads / TEAM) + (int)threadIdx.x / TEAM;
    if (TEAM < 256 && m >= a.M) return;  // larger teams have a workgroup to themselves
    const T *const x = (const T *)a.x + (int64_t)m * a.x_stride;
    const R *const residual = a.residual ? (const R *)a.residual + (int64_t)m * a.residual_stride : nullptr;
    R *const sum = (R *)a.sum + (int64_t)m * a.sum_stride;

    auto take = [&](int k) {
        f32x8 h = load_chunk<T>(x, k, K);
        if (residual) {
            h += load_chunk<R>(residual, k, K);
#pragma unroll
            for (int i = 0; i < 8; ++i) h[i] = (float)(R)h[i];
            store_chunk<R>(sum, k, K, h);
        }
        return h;
    };
    auto again = [&](int k) { return residual ? load_chunk<R>(sum, k, K) : load_chunk<T>(x, k, K); };
    double squares = 0;
    auto square = [&](f32x8 h) {
#pragma unroll
        for (int i = 0; i < 8; ++i) squares = __builtin_fma((double)h[i], (double)h[i], squares);
    };
    constexpr int kSpan = kChunks * TEAM * 8;
    f32x8 keep[kChunks];
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        keep[c] = take((c * TEAM + lane) * 8);
        square(keep[c]);
    }
    for (int k = kSpan + lane * 8; k < K; k += TEAM * 8) square(take(k));
#pragma unroll
    for (int o = 1; o < (TEAM < 64 ? TEAM : 64); o *= 2) squares += __shfl_xor(squares, o, 64);
    if constexpr (TEAM > 64) {
        if (lane % 64 == 0) squares_of[lane / 64] = squares;
        __syncthreads();
        squares = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) squares += squares_of[w];
    }
    const double r = 1.0 / __builtin_sqrt(squares / K + (double)a.eps);

    auto scaled = [&](f32x8 h, int k) {
        f32x8 w = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
        if (a.weight)
            w = a.weight_dtype == CBS_DTYPE_F32 ? load_chunk<float>((const float *)a.weight, k, K)
                                                : load_chunk<T>((const T *)a.weight, k, K);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = (float)((double)h[i] * r) * w[i];
        return h;
    };
    if constexpr (!INT8) {
        T *const y = (T *)a.y + (int64_t)m * K;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const int k = (c * TEAM + lane) * 8;
            if (k < K) store_chunk<T>(y, k, K, scaled(keep[c], k));
        }
        for (int k = kSpan + lane * 8; k < K; k += TEAM * 8) store_chunk<T>(y, k, K, scaled(again(k), k));
    } else {
        uint32_t top = 0;
        auto largest = [&](f32x8 y) {
#pragma unroll
            for (int i = 0; i < 8; ++i) top = max(top, magnitude(y[i]));
        };
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const int k = (c * TEAM + lane) * 8;
            if (k < K) {
                keep[c] = scaled(keep[c], k);
                largest(keep[c]);
            }
        }
        for (int k = kSpan + lane * 8; k < K; k += TEAM * 8) largest(scaled(again(k), k));
#pragma unroll
        for (int o = 1; o < (TEAM < 64 ? TEAM : 64); o *= 2) top = max(top, (uint32_t)__shfl_xor((int)top, o, 64));
        if constexpr (TEAM > 64) {
            if (lane % 64 == 0) top_of[lane / 64] = top;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < kWaves; ++w) top = max(top, top_of[w]);
        }
        const float s = row_scale(top), inv = row_inverse(s, top);
        auto codes = [&](f32x8 y, int k) {
            int c[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (inv != 0.f) row_codes8(y, s, inv, c);
            *(u32x2 *)(p.l.codes + ((int64_t)(k >> 6) * p.l.rows + m) * 64 + (k & 63)) =
                u32x2{pack_codes(c[0], c[1], c[2], c[3]), pack_codes(c[4], c[5], c[6], c[7])};
        };
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const int k = (c * TEAM + lane) * 8;
            if (k < p.l.Kp) codes(keep[c], k);
        }
        for (int k = kSpan + lane * 8; k < p.l.Kp; k += TEAM * 8)
            codes(k < K ? scaled(again(k), k) : f32x8{0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, k);
        if (lane == 0) p.l.scales[m] = s;
    }
}

template <typename T, typename R, int TEAM, bool INT8> hipError_t launch4(const NormArgs &a, const CodesLayout &l, hipStream_t st) {
    constexpr int kThreads = TEAM < 256 ? 256 : TEAM, kRows = kThreads / TEAM;
    // one launch but for the largest sizes: a launch holds fewer than 2^32 threads
    constexpr int kMost = 1 << 21;
    hipError_t e = hipSuccess;
    for (int m0 = 0; m0 < a.M && e == hipSuccess; m0 += kMost) {
        const NormParams p{a, l, m0};
        add_rms_norm<T, R, TEAM, INT8><<<(unsigned)((std::min(kMost, a.M - m0) + kRows - 1) / kRows), kThreads, 0, st>>>(p);
        e = hipGetLastError();
    }
    return e;
}
template <typename T, typename R, bool INT8> hipError_t launch3(const NormArgs &a, const CodesLayout &l, hipStream_t st) {
    if (a.K <= 512) return launch4<T, R, 16, INT8>(a, l, st);
    if (a.K <= 2048) return launch4<T, R, 64, INT8>(a, l, st);
    if (a.K <= 8192) return launch4<T, R, 256, INT8>(a, l, st);
    return launch4<T, R, 512, INT8>(a, l, st);
}
template <typename T, typename R> hipError_t launch2(const NormArgs &a, hipStream_t st) {
    if (a.int8) return launch3<T, R, true>(a, codes_layout(a.y, a.M, a.K), st);
    return launch3<T, R, false>(a, CodesLayout{}, st);
}
template <typename T> hipError_t launch1(const NormArgs &a, hipStream_t st) {
    return a.residual && a.residual_dtype != a.dtype ? launch2<T, float>(a, st) : launch2<T, T>(a, st);
}

}  // namespace

hipError_t launch_add_rms_norm(const NormArgs &a, hipStream_t st) {
    switch (a.dtype) {
        case CBS_DTYPE_F32: return launch2<float, float>(a, st);
        case CBS_DTYPE_BF16: return launch1<__bf16>(a, st);
        default: return launch1<_Float16>(a, st);
    }
}

}  // namespace cbs
