// k_int8_quant.hip -- the rows of the linear layer's input to 8 bits.
//
// Codes are laid out in blocks of 64 along K: code (m, k) at
// ((k / 64) * rows + m) * 64 + k % 64, with K padded by zero codes to whole
// 128s, so that the matrix kernels read the fragments of neighbouring rows as
// contiguous memory and never see past K.
//
// Bound by HBM (reads e M K bytes, writes M K).  A row is held in registers
// between finding its largest magnitude and quantising it, 32 values a lane:
// one wave per row up to K = 2048, a workgroup of four waves beyond; rows longer
// than 8192 are read a second time (from L2).  8192 x 8192 bf16: 47 to 50 us, 4.2 TB/s; a
// few rows: 4 us, the latency of one pass.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "b8_device.h"
#include "b8_linear.h"

namespace cbs {
namespace {

constexpr int kThreads = 256;
constexpr int kChunks = 4;  // of 8 values a lane keeps
constexpr int kMostRows = 1 << 22;  // of x to a launch, and workgroups that copy w

template <typename T> __device__ __forceinline__ f32x8 load_chunk(const T *row, int k, int K) {
    f32x8 x = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (k + 8 <= K) return Value<T>::load8(row + k);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (k + i < K) x[i] = Value<T>::load1(row + k + i);
    return x;
}
__device__ __forceinline__ uint32_t chunk_max(f32x8 x) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, magnitude(x[i]));
    return m;
}
__device__ __forceinline__ void store_chunk(int8_t *codes, int rows, int m, int k, f32x8 x, float s, float inv) {
    int c[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (inv != 0.f) row_codes8(x, s, inv, c);
    *(u32x2 *)(codes + ((int64_t)(k >> 6) * rows + m) * 64 + (k & 63)) =
        u32x2{pack_codes(c[0], c[1], c[2], c[3]), pack_codes(c[4], c[5], c[6], c[7])};
}

// Where the rows of w start at odd bytes, the tile kernels want them Kp apart: workgroups
// beyond those of x copy them, 16 bytes a lane.
struct Beside {
    int own;  // workgroups that have rows of x
    const int8_t *w;
    int8_t *to;
    int N;
    int64_t first;  // 16-byte piece of the copy that they begin with
    int *zeros;     // cleared by the first workgroup
    int count;
};

// TEAM lanes per row: 64 or 256.
template <typename T, int TEAM>
__global__ __launch_bounds__(kThreads) void quant_rows(const T *__restrict__ x, int64_t x_stride, int M, int K, int Kp,
                                                       int rows, int8_t *__restrict__ codes,
                                                       float *__restrict__ scales, const Beside beside) {
    __shared__ uint32_t part[4];
    if (blockIdx.x == 0)
        for (int i = (int)threadIdx.x; i < beside.count; i += kThreads) beside.zeros[i] = 0;
    if ((int)blockIdx.x >= beside.own) {
        const int64_t i = beside.first + (int64_t)((int)blockIdx.x - beside.own) * kThreads + threadIdx.x, n = i / (Kp / 16);
        const int k = (int)(i - n * (Kp / 16)) * 16;
        if (n < beside.N) *(i32x4 *)(beside.to + n * Kp + k) = load_end(beside.w, n * K + k, (int64_t)beside.N * K);
        return;
    }
    const int m = (int)blockIdx.x * (kThreads / TEAM) + (int)threadIdx.x / TEAM;
    const int lane = (int)threadIdx.x % TEAM;
    if (TEAM == 64 && m >= M) return;  // with TEAM 256 there is one workgroup per row
    const T *row = x + (int64_t)m * x_stride;
    constexpr int kSpan = kChunks * TEAM * 8;
    f32x8 keep[kChunks];
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        keep[c] = load_chunk<T>(row, (c * TEAM + lane) * 8, K);
        top = max(top, chunk_max(keep[c]));
    }
    for (int k = kSpan + lane * 8; k < K; k += TEAM * 8) top = max(top, chunk_max(load_chunk<T>(row, k, K)));
#pragma unroll
    for (int o = 1; o < 64; o *= 2) top = max(top, (uint32_t)__shfl_xor((int)top, o, 64));
    if constexpr (TEAM == 256) {
        if (lane % 64 == 0) part[lane / 64] = top;
        __syncthreads();
        top = max(max(part[0], part[1]), max(part[2], part[3]));
    }
    const float s = row_scale(top), inv = row_inverse(s, top);
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        const int k = (c * TEAM + lane) * 8;
        if (k < Kp) store_chunk(codes, rows, m, k, keep[c], s, inv);
    }
    for (int k = kSpan + lane * 8; k < Kp; k += TEAM * 8)
        store_chunk(codes, rows, m, k, load_chunk<T>(row, k, K), s, inv);
    if (lane == 0) scales[m] = s;
}

template <typename T>
hipError_t launch1(const LinearArgs &a, const CodesLayout &l, int8_t *to, int *zeros, int count, hipStream_t st) {
    const int64_t pieces = to ? (int64_t)a.N * (l.Kp / 16) : 0;
    // one launch but for the largest sizes: a launch holds fewer than 2^32 threads
    int64_t piece = 0;
    for (int m0 = 0; m0 < a.M || piece < pieces; m0 += kMostRows) {
        const T *x = (const T *)a.x + m0 * a.x_stride;
        int8_t *const codes = l.codes + (int64_t)m0 * 64;
        const int rows = std::max(0, std::min(kMostRows, a.M - m0)), own = a.K <= 2048 ? (rows + 3) / 4 : rows;
        const int copies = (int)std::min<int64_t>(kMostRows, (pieces - piece + kThreads - 1) / kThreads);
        const Beside beside{own, a.w, to, a.N, piece, zeros, zeros && m0 == 0 ? count : 0};
        if (a.K <= 2048)
            quant_rows<T, 64><<<(unsigned)(own + copies), kThreads, 0, st>>>(x, a.x_stride, rows, a.K, l.Kp, l.rows, codes,
                                                                             l.scales + m0, beside);
        else
            quant_rows<T, 256><<<(unsigned)(own + copies), kThreads, 0, st>>>(x, a.x_stride, rows, a.K, l.Kp, l.rows, codes,
                                                                              l.scales + m0, beside);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        piece += (int64_t)copies * kThreads;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_beside_rows(const LinearArgs &a, const CodesLayout &l, int8_t *to, int *zeros, int count, hipStream_t st) {
    const int64_t pieces = to ? (int64_t)a.N * (l.Kp / 16) : 0;
    int64_t piece = 0;
    do {
        const int copies = (int)std::min<int64_t>(kMostRows, (pieces - piece + kThreads - 1) / kThreads);
        // with nothing to copy, N = 0 leaves the one workgroup with the zeros
        const Beside beside{0, a.w, to, to ? a.N : 0, piece, zeros, zeros && piece == 0 ? count : 0};
        quant_rows<float, 64><<<(unsigned)std::max(1, copies), kThreads, 0, st>>>(nullptr, 0, 0, a.K, l.Kp, l.rows, nullptr,
                                                                                  nullptr, beside);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        piece += (int64_t)copies * kThreads;
    } while (piece < pieces);
    return hipSuccess;
}

int64_t rows8_bytes(int64_t M, int64_t K) { return codes_layout(nullptr, M, K).bytes; }

CodesLayout codes_layout(void *workspace, int64_t M, int64_t K) {
    CodesLayout l;
    l.rows = (int)((M + 15) / 16 * 16);
    l.Kp = (int)((K + 127) / 128 * 128);
    l.scales = (float *)workspace;
    l.codes = (int8_t *)workspace + (int64_t)l.rows * 4;
    l.bytes = (int64_t)l.rows * (4 + l.Kp);
    return l;
}

hipError_t launch_quant_rows(const LinearArgs &a, const CodesLayout &l, int8_t *to, int *zeros, int count, hipStream_t st) {
    switch (a.dtype) {
        case CBS_DTYPE_F32: return launch1<float>(a, l, to, zeros, count, st);
        case CBS_DTYPE_BF16: return launch1<__bf16>(a, l, to, zeros, count, st);
        default: return launch1<_Float16>(a, l, to, zeros, count, st);
    }
}

}  // namespace cbs
