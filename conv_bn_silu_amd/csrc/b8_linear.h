// b8_linear.h -- what the kernels of the 8-bit linear layer share: the layout of
// the quantised input in the workspace, and the epilogue.
#pragma once

#include "b8_launch.h"

#ifdef __HIPCC__
#include "b8_device.h"
#endif

namespace cbs {

// Codes of x in the workspace: scales[rows], then codes in blocks of 64 along K,
// [Kp / 64][rows][64], rows = M up to whole 16s (codes of the rows past M are
// not written and their products not stored) and Kp = K up to whole 128s.
struct CodesLayout {
    float *scales;
    int8_t *codes;
    int rows, Kp;
    int64_t bytes;
};
CodesLayout codes_layout(void *workspace, int64_t M, int64_t K);
// Quantises x; with `to`, also lays the rows of w out there, Kp apart; with `zeros`, also
// clears `count` numbers there.
hipError_t launch_quant_rows(const LinearArgs &a, const CodesLayout &l, int8_t *to, int *zeros, int count, hipStream_t st);
// The latter two alone.
hipError_t launch_beside_rows(const LinearArgs &a, const CodesLayout &l, int8_t *to, int *zeros, int count, hipStream_t st);

#ifdef __HIPCC__
// 16 bytes of w at byte `at`, some or all of which may lie past its `size` bytes: those
// come as zero and are not read.
__device__ __forceinline__ i32x4 load_end(const int8_t *w, int64_t at, int64_t size) {
    if (at + 16 <= size) return __builtin_bit_cast(i32x4, ((const Any16 *)(w + at))->v);
    uint64_t lo = 0, hi = 0;
#pragma unroll 1
    for (int64_t i = size - 1; i >= at; --i) {
        hi = hi << 8 | lo >> 56;
        lo = lo << 8 | (uint8_t)w[i];
    }
    return i32x4{(int)lo, (int)(lo >> 32), (int)hi, (int)(hi >> 32)};
}

// y = act(sum * sw * sa + bias).  The sum is exact in 32-bit integers; as fp32 it
// is rounded once (2^-24), then two products and the bias.  The weight's scale
// goes first: the row's may be as small or large as fp32 holds, and their
// product with a moderate number leaves the range only where the result does.
// e^-v = 2^(-v log2 e): the exponent's rounding costs |v| 2^-24, which 16-bit
// outputs hide and fp32 ones do not, so there the rounding is made up for.
template <typename T, bool SILU>
__device__ __forceinline__ float linear_epilogue(int sum, float sa, float sw, float bias) {
    const float v = __builtin_fmaf((float)sum * sw, sa, bias);
    if constexpr (!SILU) return v;
    constexpr float kLog2e = 1.4426950408889634f, kLog2eLow = 1.925963033500116e-8f, kLn2 = 0.6931471805599453f;
    const float h = v * -kLog2e;
    float e = __builtin_amdgcn_exp2f(h);
    if constexpr (sizeof(T) == 4) {
        const float low = __builtin_fmaf(v, -kLog2e, -h) - v * kLog2eLow;
        if (fabsf(h) < 126.f) e = __builtin_fmaf(e, low * kLn2, e);
    }
    return v * __builtin_amdgcn_rcpf(1.0f + e);
}
#endif

}  // namespace cbs
