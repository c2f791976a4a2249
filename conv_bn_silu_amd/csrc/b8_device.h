// b8_device.h -- device-side helpers shared by the kernels of the 8-bit block
// operators: element types, wave reductions and rows to 8 bits.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "cbs_device.h"

namespace cbs {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x16 __attribute__((ext_vector_type(16)));
typedef float f32x8 __attribute__((ext_vector_type(8)));

// 16 bytes at any address: the memory path serves them as one access whatever the
// alignment, so that one kernel does for tensors at multiples of 16 bytes and others.
struct __attribute__((packed, aligned(1))) Any16 {
    u32x4 v;
};

// Value types of the operators' inputs and outputs, 8 elements at a time or one (for
// ragged ends).  Stores round to nearest even.
template <typename T> struct Value {
    typedef T x8 __attribute__((ext_vector_type(8)));
    static __device__ __forceinline__ float load1(const T *p) { return (float)*p; }
    static __device__ __forceinline__ void store1(T *p, float v) { *p = (T)v; }
    static __device__ __forceinline__ f32x8 load8(const T *p) {
        return __builtin_convertvector(__builtin_bit_cast(x8, ((const Any16 *)p)->v), f32x8);
    }
    static __device__ __forceinline__ void store8(T *p, f32x8 v) {
        ((Any16 *)p)->v = __builtin_bit_cast(u32x4, __builtin_convertvector(v, x8));
    }
};
template <> struct Value<float> {
    static __device__ __forceinline__ float load1(const float *p) { return *p; }
    static __device__ __forceinline__ void store1(float *p, float v) { *p = v; }
    static __device__ __forceinline__ f32x8 load8(const float *p) {
        const f32x4 a = __builtin_bit_cast(f32x4, ((const Any16 *)p)[0].v), b = __builtin_bit_cast(f32x4, ((const Any16 *)p)[1].v);
        return f32x8{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    }
    static __device__ __forceinline__ void store8(float *p, f32x8 v) {
        ((Any16 *)p)[0].v = __builtin_bit_cast(u32x4, f32x4{v[0], v[1], v[2], v[3]});
        ((Any16 *)p)[1].v = __builtin_bit_cast(u32x4, f32x4{v[4], v[5], v[6], v[7]});
    }
};

// Rows to 8 bits.  The largest magnitude is taken on the bit patterns without
// sign, so that a NaN (above infinity) is not lost.
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// The scale of a row whose largest magnitude has these bits: fp32(amax / 127),
// at least the smallest normal number; infinity and NaN stay.
__device__ __forceinline__ float row_scale(uint32_t amax_bits) {
    const float amax = __uint_as_float(amax_bits);
    if (amax_bits > 0x7F800000u) return amax;
    return fmaxf(__fdiv_rn(amax, 127.f), 0x1p-126f);
}

// Codes of 8 values of a row of scale s (inv = 1 / s to within 2 ulp): the
// nearest integers to x / s, ties to even.  x * inv is off by less than 4e-5, so
// its nearest integer is right unless it lies that close to a border between
// two codes.  Only then is the remainder x - n s looked at, which fma gives
// exactly: with |n| >= 1 it is a multiple of half an ulp of s and below s.
__device__ __forceinline__ void row_codes8(f32x8 x, float s, float inv, int (&code)[8]) {
    float far = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float q = x[i] * inv, n = __builtin_rintf(q);
        far = fmaxf(far, fabsf(q - n));
        code[i] = (int)n;
    }
    if (__builtin_expect(far > 0.4999f, 0)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float n = (float)code[i];
            const float r2 = 2.f * __builtin_fmaf(-n, s, x[i]);
            const bool odd = (code[i] & 1) != 0;
            if (r2 > s || (r2 == s && odd)) n += 1.f;
            else if (r2 < -s || (r2 == -s && odd)) n -= 1.f;
            code[i] = (int)n;
        }
    }
}
__device__ __forceinline__ uint32_t pack_codes(int a, int b, int c, int d) {
    return (uint32_t)(a & 255) | (uint32_t)(b & 255) << 8 | (uint32_t)(c & 255) << 16 | (uint32_t)d << 24;
}
// A scale that takes part in no quotient: rows that hold an infinity or a NaN get codes 0.
__device__ __forceinline__ float row_inverse(float s, uint32_t amax_bits) {
    return amax_bits >= 0x7F800000u ? 0.f : __fdiv_rn(1.f, s);
}

}  // namespace cbs
