// k_norm.hip -- the residual's addition with the root-mean-square norm:
// h = x + residual, y = h w / sqrt(mean(h^2) + eps), y in x's type or as rows in 8 bits.
//
// Bound by HBM: x and the residual are read once, h and y written once, and a row stays in
// registers in between.  8 values a lane, and as many lanes as the row has 8s: many short workgroups, each with
// one access of a tensor a lane on its way, draw the most (16384 x 8192, bf16 with residual: 256 lanes with 32
// values each 203 us, 512 with 16 207, 1024 with 8 180; 1.07 GB at the rate of a large copy, 6.3 TB/s: 170).
// Rows beyond 8192 take 16 values a lane, those beyond 16384 read h a second time.  What the memory-side cache cannot
// hold passes by the caches (180 -> 170 us; outputs in 8 bits stay, for the layer reads them: 8192 x 8192 with
// what is read passing by as well 220 us into a layer of 1024, without 214), and eight workgroups of neighbouring rows
// share an XCD (172 -> 169).  Together 171 us, 6.3 TB/s.
//   Rows of 1024 (131072 of them) 170 us for 170, of 256 (300000) 98 for 98, of 128 (a million, no residual) 87
//   for 85; 16384 wide 174 for 170; 32768 wide 207 for 170; one row of 4096: 2.3 us on the GPU, 5 to 6 a call.
//   Widths in no whole 8s are guarded access by access and do not pass by the caches: 8191 wide 294 for 170.
// With 8 bits the vector unit counts as well (451 instructions for a lane's 8 values at first, 87% of the cycles, 413
// and 85% now): sizes of whole 8s have no ragged ends, and codes come out of one fused addition each.  8192 x 8192, bf16 with
// residual: 104 -> 94 us (470 MB: 75), of 16384 253 -> 170 (149); residual in fp32 127 (738 MB: 117); 8191 wide 170 (75).
//
// Squares are summed in 64 bits: no row of finite numbers overflows or vanishes on the way.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "b8_device.h"
#include "b8_linear.h"
#include "st_device.h"
#include "st_launch.h"

namespace cbs {
namespace {

struct NormParams {
    NormArgs a;
    CodesLayout l;  // of y in 8 bits
    int m0;         // row that the launch begins with
    double inv_k;   // 1 / K
};

// 1 / sqrt(s) for s > 0: the instruction is good to 2^-23, one step of Newton's doubles the bits.
__device__ __forceinline__ double reciprocal_root(double s) {
    const double r = __builtin_amdgcn_rsq(s), better = __builtin_fma(0.5 * r, __builtin_fma(-s * r, r, 1.0), r);
    return s == INFINITY ? 0.0 : better;
}

// 8 values of a row from k on.  FULL: K is a whole number of 8s, so that nothing is ragged (what is does not stream).
template <bool FULL, bool STREAM, typename T> __device__ __forceinline__ Held<T> take(const T *row, int k, int K) {
    if constexpr (FULL) return k < K ? Held<T>::template load<STREAM>(row + k) : Held<T>{};
    else return Held<T>(load_chunk(row, k, K));
}
template <bool FULL, bool STREAM, typename T> __device__ __forceinline__ void put(T *row, int k, int K, const Held<T> &v) {
    if constexpr (FULL) v.template store<STREAM>(row + k);
    else v.store_chunk(row, k, K);
}

// 8 weights on their way: they are asked for before the sum of squares, and wanted after it.  Wide ones beside
// narrow values are not, for the registers they take would cost more than the wait.
template <typename T, bool FULL> struct Weights {
    Held<T> held;
    __device__ __forceinline__ void load(const NormArgs &a, int k) {
        if (a.weight && a.weight_dtype == a.dtype) held = take<FULL, false>((const T *)a.weight, k, a.K);
    }
    __device__ __forceinline__ f32x8 get(const NormArgs &a, int k) const {
        if (!a.weight) return f32x8{1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
        return a.weight_dtype == a.dtype ? held.get() : take<FULL, false>((const float *)a.weight, k, a.K).get();
    }
};

// T: type of x and y, R: of the residual and the sum.  TEAM lanes to a row; teams of 128 and less share a
// workgroup of 256, or a row has a workgroup (TEAM 0).  CHUNKS: of 8 values a lane keeps.  STREAM: the tensors pass by
// the caches.
template <typename T, typename R, int TEAM, int CHUNKS, bool INT8, bool FULL, bool STREAM>
__global__ __launch_bounds__(TEAM ? 256 : 1024) void add_rms_norm(const NormParams p) {
    constexpr int kLanes = TEAM == 0 || TEAM > 64 ? 64 : TEAM, kMostWaves = TEAM ? 4 : 16;
    constexpr bool kMeet = TEAM == 0 || TEAM > 64;  // a row's waves meet in LDS
    constexpr bool kOnce = STREAM && !INT8;
    __shared__ double squares_of[kMostWaves];
    __shared__ uint32_t top_of[kMostWaves];
    const NormArgs &a = p.a;
    const int team = TEAM ? TEAM : (int)blockDim.x, tid = (int)threadIdx.x, lane = TEAM ? tid % TEAM : tid, K = a.K;
    // workgroups go to the eight XCDs in turn; of 64, each gets 8 with rows side by side
    const int id = (int)blockIdx.x, group = id & ~63, in = id & 63;
    const int place = group + 64 <= (int)gridDim.x ? group + in % 8 * 8 + in / 8 : id;
    int m = p.m0 + (TEAM ? place * (256 / team) + tid / team : place);
    const bool mine = TEAM == 0 || m < a.M;
    if (!kMeet && !mine) return;
    if (TEAM) m = min(m, a.M - 1);  // reads the last row and writes nothing
    const T *const x = (const T *)a.x + (int64_t)m * a.x_stride;
    const R *const residual = a.residual ? (const R *)a.residual + (int64_t)m * a.residual_stride : nullptr;
    R *const sum = (R *)a.sum + (int64_t)m * a.sum_stride;
    const int end = mine ? K : 0, code_end = mine ? p.l.Kp : 0;  // of what is written

    auto add = [&](const Held<T> &h, const Held<R> &r, int k) {
        const Held<R> v(h.get() + r.get());
        if (k < end) put<FULL, STREAM>(sum, k, K, v);
        return v;
    };
    auto again = [&](int k) { return residual ? take<FULL, false>((const R *)sum, k, K).get() : take<FULL, false>(x, k, K).get(); };
    auto square = [&](double &to, f32x8 h) {
#pragma unroll
        for (int i = 0; i < 8; ++i) to = __builtin_fma((double)h[i], (double)h[i], to);
    };
    const int span = CHUNKS * team * 8;
    // h is a number of R's with a residual, of T's without, which R holds too
    Held<R> keep[CHUNKS];
    Weights<T, FULL> weights[CHUNKS];
    {
        Held<T> h[CHUNKS];
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) h[c] = take<FULL, kOnce>(x, (c * team + lane) * 8, K);
        if (residual) {
            Held<R> r[CHUNKS];
#pragma unroll
            for (int c = 0; c < CHUNKS; ++c) r[c] = take<FULL, kOnce>(residual, (c * team + lane) * 8, K);
#pragma unroll
            for (int c = 0; c < CHUNKS; ++c) weights[c].load(a, (c * team + lane) * 8);
#pragma unroll
            for (int c = 0; c < CHUNKS; ++c) keep[c] = add(h[c], r[c], (c * team + lane) * 8);
        } else {
#pragma unroll
            for (int c = 0; c < CHUNKS; ++c) weights[c].load(a, (c * team + lane) * 8);
#pragma unroll
            for (int c = 0; c < CHUNKS; ++c) keep[c] = Held<R>(h[c].get());
        }
    }
    double part[CHUNKS] = {}, squares = 0;
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) square(part[c], keep[c].get());
    for (int k = span + lane * 8; k < K; k += team * 8) {
        const Held<T> h = take<FULL, false>(x, k, K);
        square(squares, residual ? add(h, take<FULL, false>(residual, k, K), k).get() : h.get());
    }
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) squares += part[c];
    squares = team_sum<kLanes>(squares);
    // a row's waves, and this lane's of them where they meet
    const int waves = team / 64, wave0 = TEAM == 128 ? tid / 128 * 2 : 0, its = wave0 + tid % (TEAM ? 2 : 16);
    const bool there = its < wave0 + waves;
    if constexpr (kMeet) {
        if (tid % 64 == 0) squares_of[tid / 64] = squares;
        __syncthreads();
        squares = team_sum<TEAM ? 2 : 16>(there ? squares_of[its] : 0.0);
    }
    // h r in fp32 with one rounding: r in two parts, and where it comes near fp32's smallest numbers h and r
    // meet half way
    double r = reciprocal_root(__builtin_fma(squares, p.inv_k, (double)a.eps));
    const bool small = r < 0x1p-64;
    if (small) r *= 0x1p64;
    const float r_hi = (float)r, r_lo = (float)(r - (double)r_hi);
    auto scaled = [&](f32x8 h, f32x8 w) {
        if (__builtin_expect(small, 0)) h *= 0x1p-64f;
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = __builtin_fmaf(h[i], r_hi, h[i] * r_lo) * w[i];
        return h;
    };
    auto scaled_again = [&](int k) {
        Weights<T, FULL> w;
        w.load(a, k);
        return scaled(again(k), w.get(a, k));
    };
    if constexpr (!INT8) {
        T *const y = (T *)a.y + (int64_t)m * K;
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) {
            const int k = (c * team + lane) * 8;
            if (k < end) put<FULL, STREAM>(y, k, K, Held<T>(scaled(keep[c].get(), weights[c].get(a, k))));
        }
        for (int k = span + lane * 8; k < end; k += team * 8) put<FULL, STREAM>(y, k, K, Held<T>(scaled_again(k)));
    } else {
        uint32_t top = 0;
        auto largest = [&](f32x8 y) {
#pragma unroll
            for (int i = 0; i < 8; ++i) top = max(top, magnitude(y[i]));
        };
        // two chunks are scaled twice: kept, they would cost the registers of a second workgroup on the CU
        f32x8 y = {};
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) {
            const int k = (c * team + lane) * 8;
            if (k < K) {
                y = scaled(keep[c].get(), weights[c].get(a, k));
                largest(y);
            }
        }
        for (int k = span + lane * 8; k < end; k += team * 8) largest(scaled_again(k));
        top = team_max_of<kLanes>(top);
        if constexpr (kMeet) {
            if (tid % 64 == 0) top_of[tid / 64] = top;
            __syncthreads();
            top = team_max_of<TEAM ? 2 : 16>(there ? top_of[its] : 0u);
        }
        const float s = row_scale(top), inv = row_quotient(s, top);
        auto codes = [&](f32x8 y, int k) {
            *(u32x2 *)(p.l.codes + ((int64_t)(k >> 6) * p.l.rows + m) * 64 + (k & 63)) = inv != 0.f ? codes_of8(y, s, inv) : u32x2{0u, 0u};
        };
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) {
            const int k = (c * team + lane) * 8;
            if (CHUNKS > 1) y = k < K ? scaled(keep[c].get(), weights[c].get(a, k)) : f32x8{};
            if (k < code_end) codes(y, k);
        }
        for (int k = span + lane * 8; k < code_end; k += team * 8)
            codes(k < K ? scaled_again(k) : f32x8{0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, k);
        if (lane == 0 && mine) p.l.scales[m] = s;
    }
}

template <typename T, typename R, int TEAM, int CHUNKS, bool INT8, bool FULL, bool STREAM>
hipError_t launch5(const NormArgs &a, const CodesLayout &l, hipStream_t st) {
    const int rows = TEAM ? 256 / TEAM : 1, threads = TEAM ? 256 : std::min(1024, (a.K + 512 * CHUNKS - 1) / (512 * CHUNKS) * 64);
    // one launch but for the largest sizes: a launch holds fewer than 2^32 threads
    constexpr int kMost = 1 << 21;
    hipError_t e = hipSuccess;
    for (int m0 = 0; m0 < a.M && e == hipSuccess; m0 += kMost) {
        const NormParams p{a, l, m0, 1.0 / a.K};
        const unsigned grid = (unsigned)((std::min(kMost, a.M - m0) + rows - 1) / rows);
        add_rms_norm<T, R, TEAM, CHUNKS, INT8, FULL, STREAM><<<grid, threads, 0, st>>>(p);
        e = hipGetLastError();
    }
    return e;
}
template <typename T, typename R, int TEAM, int CHUNKS, bool INT8> hipError_t launch4(const NormArgs &a, const CodesLayout &l, hipStream_t st) {
    if (a.K % 8 != 0) return launch5<T, R, TEAM, CHUNKS, INT8, false, false>(a, l, st);
    const int64_t bytes = (int64_t)a.M * a.K * ((a.int8 ? 1 : 2) * sizeof(T) + (a.residual ? 2 * sizeof(R) : 0));
    return bytes > kCached ? launch5<T, R, TEAM, CHUNKS, INT8, true, true>(a, l, st) : launch5<T, R, TEAM, CHUNKS, INT8, true, false>(a, l, st);
}
template <typename T, typename R, bool INT8> hipError_t launch3(const NormArgs &a, const CodesLayout &l, hipStream_t st) {
    if (a.K <= 128) return launch4<T, R, 16, 1, INT8>(a, l, st);
    if (a.K <= 256) return launch4<T, R, 32, 1, INT8>(a, l, st);
    if (a.K <= 512) return launch4<T, R, 64, 1, INT8>(a, l, st);
    if (a.K <= 1024) return launch4<T, R, 128, 1, INT8>(a, l, st);
    if (a.K <= 8192) return launch4<T, R, 0, 1, INT8>(a, l, st);
    return launch4<T, R, 0, 2, INT8>(a, l, st);
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
