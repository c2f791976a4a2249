// st_device.h -- sums, maxima and running sums over neighbouring lanes, by the vector unit's own lane
// exchanges: a step is one or two instructions, where one through LDS takes some hundred cycles.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "b8_device.h"

namespace cbs {

constexpr int64_t kCached = 256 << 20;  // bytes that the memory-side cache holds

// 16 bytes at any address, of tensors that are read and written once: they take no room in the caches that others want.
struct Streamed {
    typedef u32x4 __attribute__((aligned(1))) any;
    static __device__ __forceinline__ u32x4 load(const void *p) { return __builtin_nontemporal_load((const any *)p); }
    static __device__ __forceinline__ void store(void *p, u32x4 v) { __builtin_nontemporal_store(v, (any *)p); }
};

// 8 values from k on, zeros from K on.
template <typename T> __device__ __forceinline__ f32x8 load_chunk(const T *row, int k, int K) {
    f32x8 x = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (k + 8 <= K) return Value<T>::load8(row + k);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (k + i < K) x[i] = Value<T>::load1(row + k + i);
    return x;
}

// 8 values as T holds them.
template <typename T> struct Held {
    u32x4 raw[sizeof(T) / 2];
    Held() = default;
    template <bool STREAM> static __device__ __forceinline__ Held load(const T *p) {
        Held h;
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i)
            h.raw[i] = STREAM ? Streamed::load((const char *)p + 16 * i) : ((const Any16 *)p)[i].v;
        return h;
    }
    __device__ __forceinline__ explicit Held(f32x8 v) {
        if constexpr (sizeof(T) == 4) {
            raw[0] = __builtin_bit_cast(u32x4, f32x4{v[0], v[1], v[2], v[3]});
            raw[1] = __builtin_bit_cast(u32x4, f32x4{v[4], v[5], v[6], v[7]});
        } else {
            raw[0] = __builtin_bit_cast(u32x4, __builtin_convertvector(v, typename Value<T>::x8));
        }
    }
    __device__ __forceinline__ f32x8 get() const {
        if constexpr (sizeof(T) == 4) {
            const f32x4 a = __builtin_bit_cast(f32x4, raw[0]), b = __builtin_bit_cast(f32x4, raw[1]);
            return f32x8{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        } else {
            return __builtin_convertvector(__builtin_bit_cast(typename Value<T>::x8, raw[0]), f32x8);
        }
    }
    template <bool STREAM> __device__ __forceinline__ void store(T *p) const {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
            if constexpr (STREAM) Streamed::store((char *)p + 16 * i, raw[i]);
            else ((Any16 *)p)[i].v = raw[i];
        }
    }
    // To row[k ..], as far as K.
    __device__ __forceinline__ void store_chunk(T *row, int k, int K) const {
        if (k + 8 <= K) return store<false>(row + k);
        const f32x8 v = get();
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (k + i < K) Value<T>::store1(row + k + i, v[i]);
    }
};

// The value of the lane that the control names; `old` where there is none or the mask leaves the row out.
template <int CTRL, int ROWS = 15> __device__ __forceinline__ uint32_t lane_from(uint32_t old, uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp((int)old, (int)v, CTRL, ROWS, 15, false);
}
constexpr int kSwap1 = 0xB1, kSwap2 = 0x4E, kMirror8 = 0x141, kMirror16 = 0x140;  // within 4, 4, 8, 16 lanes

// Combines a value over teams of TEAM consecutive lanes (a power of two up to 64), in every lane of them.  `f`
// takes the value and the word-wise exchange, and returns the value combined with its exchanged self.  Values of
// equal smaller teams are equal, so that mirrors serve as well as shifts.
template <int TEAM, typename T, typename F> __device__ __forceinline__ T over_team(T v, F &&f) {
    if constexpr (TEAM > 1) v = f(v, [](uint32_t a) { return lane_from<kSwap1>(a, a); });
    if constexpr (TEAM > 2) v = f(v, [](uint32_t a) { return lane_from<kSwap2>(a, a); });
    if constexpr (TEAM > 4) v = f(v, [](uint32_t a) { return lane_from<kMirror8>(a, a); });
    if constexpr (TEAM > 8) v = f(v, [](uint32_t a) { return lane_from<kMirror16>(a, a); });
    const int lane = (int)__lane_id();
    if constexpr (TEAM > 16)
        v = f(v, [lane](uint32_t a) {
            const auto r = __builtin_amdgcn_permlane16_swap(a, a, false, false);
            return (uint32_t)(lane & 16 ? r[0] : r[1]);
        });
    if constexpr (TEAM > 32)
        v = f(v, [lane](uint32_t a) {
            const auto r = __builtin_amdgcn_permlane32_swap(a, a, false, false);
            return (uint32_t)(lane & 32 ? r[0] : r[1]);
        });
    return v;
}
template <int TEAM> __device__ __forceinline__ uint32_t team_max_of(uint32_t v) {
    return over_team<TEAM>(v, [](uint32_t a, auto &&other) { return max(a, other(a)); });
}
template <int TEAM> __device__ __forceinline__ double team_sum(double v) {
    return over_team<TEAM>(v, [](double a, auto &&other) {
        const uint64_t w = __builtin_bit_cast(uint64_t, a);
        return a + __builtin_bit_cast(double, (uint64_t)other((uint32_t)(w >> 32)) << 32 | other((uint32_t)w));
    });
}

template <int TEAM> __device__ __forceinline__ uint32_t team_sum_of(uint32_t v) {
    return over_team<TEAM>(v, [](uint32_t a, auto &&other) { return a + other(a); });
}

// A row's factor of the quotients, by the instruction's reciprocal (good to 1 ulp, which is enough for the codes); 0
// where the row holds an infinity or a NaN and gets the codes 0.
__device__ __forceinline__ float row_quotient(float s, uint32_t amax_bits) {
    return amax_bits >= 0x7F800000u ? 0.f : __builtin_amdgcn_rcpf(s);
}

// Codes of 8 values of a row as row_codes8 (b8_device.h) has them, packed, in fewer instructions: adding 1.5 2^23 leaves
// the nearest whole number to x inv, ties to even, in the sum's low bits, and the distance from it says whether x lies
// so near a border that the remainder has to be looked at.  For |x inv| below 2^21 (or no number at all).
__device__ __forceinline__ u32x2 codes_of8(f32x8 x, float s, float inv) {
    constexpr float kWhole = 12582912.f;
    uint32_t t[8];
    float far = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float sum = __builtin_fmaf(x[i], inv, kWhole);
        t[i] = __float_as_uint(sum);
        far = fmaxf(far, fabsf(__builtin_fmaf(x[i], inv, kWhole - sum)));
    }
    if (__builtin_expect(far > 0.4999f, 0)) {
        int c[8];
        row_codes8(x, s, inv, c);
        return u32x2{pack_codes(c[0], c[1], c[2], c[3]), pack_codes(c[4], c[5], c[6], c[7])};
    }
    // the low bytes of two words, side by side
    auto two = [](uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x0C0C0400u); };
    auto four = [](uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x05040100u); };
    return u32x2{four(two(t[0], t[1]), two(t[2], t[3])), four(two(t[4], t[5]), two(t[6], t[7]))};
}

// Sums over the lanes of a 16, or of the wave, up to this one, which do not pass `most` (below 2^31).
__device__ __forceinline__ uint32_t sixteen_upto(uint32_t v, uint32_t most) {
    v = min(v, most);
    v = min(v + lane_from<0x111>(0, v), most);  // from 1 lane before,
    v = min(v + lane_from<0x112>(0, v), most);  // 2,
    v = min(v + lane_from<0x114>(0, v), most);  // 4
    return min(v + lane_from<0x118>(0, v), most);  // and 8
}
__device__ __forceinline__ uint32_t lanes_upto(uint32_t v, uint32_t most) {
    v = sixteen_upto(v, most);
    v = min(v + lane_from<0x142, 0xA>(0, v), most);  // the last of the 16 before, to the second and the fourth
    return min(v + lane_from<0x143, 0xC>(0, v), most);  // the last of the first 32, to the others
}

}  // namespace cbs
