// k_int8_linear.hip -- the product of the linear layer in 8-bit integers and its
// epilogue.
#include <hip/hip_runtime.h>

#include "b8_device.h"
#include "b8_linear.h"

namespace cbs {
namespace {

constexpr int kThreads = 256;
constexpr int kPitch = 80;  // bytes of a 64-byte row in LDS, off the bank period

// 64 x 64 outputs per workgroup, 4 x 4 a lane, 64 of K at a time through LDS.
template <typename T, bool SILU>
__global__ __launch_bounds__(kThreads) void linear_tile(const CodesLayout l, const int8_t *__restrict__ w,
                                                        const float *__restrict__ w_scale,
                                                        const float *__restrict__ bias, T *__restrict__ y, int M, int N,
                                                        int K) {
    __shared__ __attribute__((aligned(16))) int8_t as[64 * kPitch], bs[64 * kPitch];
    const int m0 = (int)blockIdx.y * 64, n0 = (int)blockIdx.x * 64, t = (int)threadIdx.x;
    const int tm = t / 16, tn = t % 16;
    int acc[4][4] = {};
    for (int k0 = 0; k0 < l.Kp; k0 += 64) {
        const int r = t / 4, c = t % 4 * 16;
        const int m = min(m0 + r, l.rows - 1);
        *(i32x4 *)(as + r * kPitch + c) = *(const i32x4 *)(l.codes + ((int64_t)(k0 / 64) * l.rows + m) * 64 + c);
        const int8_t *wr = w + (int64_t)min(n0 + r, N - 1) * K + k0 + c;
        for (int i = 0; i < 16; ++i) bs[r * kPitch + c + i] = k0 + c + i < K ? wr[i] : (int8_t)0;
        __syncthreads();
        for (int k = 0; k < 64; k += 4) {
            int a[4], b[4];
            for (int i = 0; i < 4; ++i) a[i] = *(const int *)(as + (tm * 4 + i) * kPitch + k);
            for (int j = 0; j < 4; ++j) b[j] = *(const int *)(bs + (tn + 16 * j) * kPitch + k);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_amdgcn_sdot4(a[i], b[j], acc[i][j], false);
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int m = m0 + tm * 4 + i, n = n0 + tn + 16 * j;
            if (m < M && n < N)
                Value<T>::store1(y + (int64_t)m * N + n,
                                 linear_epilogue<T, SILU>(acc[i][j], l.scales[m], w_scale[n], bias ? bias[n] : 0.f));
        }
}

template <typename T> hipError_t launch_tile(const LinearArgs &a, const CodesLayout &l, hipStream_t st) {
    const dim3 grid((a.N + 63) / 64, (a.M + 63) / 64);
    if (a.act == CBS_ACT_SILU)
        linear_tile<T, true><<<grid, kThreads, 0, st>>>(l, a.w, a.w_scale, a.bias, (T *)a.y, a.M, a.N, a.K);
    else
        linear_tile<T, false><<<grid, kThreads, 0, st>>>(l, a.w, a.w_scale, a.bias, (T *)a.y, a.M, a.N, a.K);
    return hipGetLastError();
}

}  // namespace

int64_t linear_workspace(int64_t M, int64_t N, int64_t K) {
    (void)N;
    return codes_layout(nullptr, M, K).bytes;
}

hipError_t launch_int8_linear(const LinearArgs &a, int num_cu, hipStream_t st) {
    (void)num_cu;
    const CodesLayout l = codes_layout(a.workspace, a.M, a.K);
    const hipError_t e = launch_quant_rows(a, l, st);
    if (e != hipSuccess) return e;
    switch (a.dtype) {
        case CBS_DTYPE_F32: return launch_tile<float>(a, l, st);
        case CBS_DTYPE_BF16: return launch_tile<__bf16>(a, l, st);
        default: return launch_tile<_Float16>(a, l, st);
    }
}

}  // namespace cbs
