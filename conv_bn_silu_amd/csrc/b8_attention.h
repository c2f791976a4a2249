// b8_attention.h -- what the kernels of the paged attention share: how the work
// is divided, where a row's keys lie, and 8-bit codes as matrix operands.
//
// Rows.  The queries that read one key/value head of one sequence are its
// rows: row r is new token r / group, head r % group of the head's group, so
// that neighbouring rows see (nearly) the same keys.  A tile is some 16s of rows.
//
// Scores.  S^T = K Q^T: with keys along the rows of the matrix instruction's
// result and queries along its columns, a lane holds one query and a set of keys,
// and the softmax over keys is arithmetic within the lane but for one exchange
// at the end.  The probabilities are then, as they stand, the operand of
// O^T = V^T P^T, whose result again has one query to a lane.
//
// Bits.  Scores, maxima, sums and outputs are fp32.  What meets in a matrix instruction has 16 bits,
// for those of fp32 take 16 times as long: the probabilities are rounded to the cache's type (bf16 or
// fp16; fp16 for 8-bit codes), off by half a step of it each, while the sum adds them unrounded.  That shows: the error of
// the outputs against 64 bits is 0.0021 of their size where rounding the outputs alone would leave
// 0.0016 (bf16), 0.0003 and 0.0002 (fp16).
//
// Units.  t = q . k (times the key's scale), x = c t the exponent of two, with
// c = |scale| log2 e and the scale's sign put into q.  The running maximum m is
// one of t; a probability is 2^(c t - c m).  m moves only where a score passes it
// by more than 2^8 (probabilities then reach 256, which every type here holds), so
// that the outputs are rarely rescaled.
//
// 8-bit caches.  Codes are whole numbers below 2^11 and so exact in fp16.
// Queries in bf16 become fp16 after a power of two per row, which brings the
// row's largest to [2^14, 2^15): values down to 2^-28 of the largest stay exact, smaller
// ones are off by 2^-39 of it, below what the fp32 sum of the products loses.
// A value's scale goes into its probability, and the product, like the queries, into
// fp16 (10 bits after the point: half a step of 2^-11 of each, and what lies below 2^-24 of
// half of the row's largest product is off by up to half of that).  So that it fits whatever the scales,
// each row keeps two exponents: `m` of its largest probability, in whose unit the sum is kept, and `mo`, 2^6
// below its largest product of probability and scale, in whose unit the outputs are.  Both follow
// only what the row sees: a key behind the mask may have any scale, and so may one of negligible weight.
// Where the scales of a tile lie within 2^7 of each other (nearly always), one
// power of two above stands for all of them in mo, and goes into the exponent of the
// probabilities; else the largest product is looked for (see `ValueUnit`).
#pragma once

#include "b8_launch.h"

#ifdef __HIPCC__
#include <type_traits>

#include "b8_device.h"
#endif

namespace cbs {

// How a call is divided.  Sequences of few rows go to attend_few, the others to
// attend_many; each takes the keys of a tile `chunk` at a time by different
// workgroups.  Where a tile has more than one chunk, its parts go through the
// workspace: a maximum (as an exponent of two), a sum and an output for each row.
struct AttentionPart {
    int tile;           // rows of a tile
    int chunk, chunks;  // keys of a chunk; most chunks a tile can have
    int room;           // chunks that the workspace has room for
    float *o, *ml;      // [line][room][dim] and [line][room][2]
};
struct AttentionPlan {
    AttentionArgs a;
    FastDiv page, group;
    bool few_only;  // attend_many does not run
    bool split;     // attend_many: two waves to a row
    int slots;      // most tiles that attend_many can have
    AttentionPart few, many;
};
hipError_t launch_attend_few(const AttentionPlan &p, hipStream_t st);
hipError_t launch_attend_many(const AttentionPlan &p, hipStream_t st);
int many_tile(int64_t dim, bool int8, bool split);  // rows of its tile

#ifdef __HIPCC__
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.f;  // of the running maximum, as an exponent of two
// fp16 holds 2^(8 + 6): what meets the values in it is 2^6 times as large as the unit says, so that
// less is lost at its lower end, which small probabilities of large values reach.
constexpr float kLift = 6.f;
template <typename X> constexpr float kLiftOf = std::is_same_v<X, _Float16> ? kLift : 0.f;

struct Sequence {
    int b, first, n, len;  // its rows of q and the tokens it has in the cache
};
__device__ __forceinline__ Sequence sequence(const AttentionPlan &p, int b) {
    const int first = max(0, min(p.a.starts[b], p.a.tokens));
    const int next = max(first, min(p.a.starts[b + 1], p.a.tokens));
    return Sequence{b, first, next - first, max(0, p.a.lens[b])};
}
__device__ __forceinline__ bool is_many(const AttentionPlan &p, int rows) {
    return !p.few_only && rows > p.few.tile;
}
// First key that the token at position pos sees, of the last `window`.
__device__ __forceinline__ int first_key(const AttentionPlan &p, int pos) {
    return p.a.window == 0 ? 0 : (int)max((int64_t)0, (int64_t)pos + 1 - p.a.window);
}
// Keys [lo, hi) that the rows [r0, r1) of a sequence may see.
struct Span2 {
    int lo, hi;
};
__device__ __forceinline__ Span2 keys_of(const AttentionPlan &p, const Sequence &s, int r0, int r1) {
    const int from = s.len - s.n + (int)p.group.div((uint32_t)r0), to = s.len - s.n + (int)p.group.div((uint32_t)(r1 - 1));
    const int limit = p.a.table_width * (int)p.page.d;
    const int hi = max(0, min(to + 1, limit));
    return Span2{min(first_key(p, from), hi), hi};
}
__device__ __forceinline__ int chunks_of(const AttentionPart &part, Span2 k) {
    return max(1, (k.hi - k.lo + part.chunk - 1) / part.chunk);
}
// Where row r of a sequence lies in the output, as [token][head].
__device__ __forceinline__ int64_t out_line(const AttentionPlan &p, const Sequence &s, int kvh, int r) {
    const int tok = (int)p.group.div((uint32_t)r);
    return (int64_t)(s.first + tok) * p.a.heads + kvh * (int)p.group.d + r - tok * (int)p.group.d;
}
// Its line among the parts: with attend_many beside it, attend_few has at most a tile of a sequence.
__device__ __forceinline__ int64_t few_line(const AttentionPlan &p, const Sequence &s, int kvh, int r) {
    return p.few_only ? out_line(p, s, kvh, r) : ((int64_t)s.b * p.a.cache.heads + kvh) * p.few.tile + r;
}

// 4 codes as fp16: with the sign bit flipped, the byte below 0x64 is the fp16
// number 1024 + 128 + code.
__device__ __forceinline__ f16x4 codes_f16(uint32_t c) {
    const uint32_t u = c ^ 0x80808080u;
    const f16x2 off = {(_Float16)1152.f, (_Float16)1152.f};
    const f16x2 lo = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u)) - off;
    const f16x2 hi = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u)) - off;
    return f16x4{lo.x, lo.y, hi.x, hi.y};
}
__device__ __forceinline__ f16x8 codes_f16(uint32_t a, uint32_t b) {
    const f16x4 x = codes_f16(a), y = codes_f16(b);
    return f16x8{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
}

// Operands of the matrix instructions for a cache of type C under queries of type T:
// fp16 for 8-bit codes, else the cache's own type.
template <typename T, typename C> struct Operand {
    using type = std::conditional_t<std::is_same_v<C, int8_t>, _Float16, C>;
    typedef type x8 __attribute__((ext_vector_type(8)));
};
__device__ __forceinline__ f32x4 mma16(f16x8 a, f16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma16(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma32(f16x8 a, f16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma32(bf16x8 a, bf16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// Transposed reads of LDS: of the 4 (8) rows by 16 columns whose pieces of 8 bytes
// the 16 lanes of a group name in order, lane i gets column i.
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ u32x2 read_tr16(const unsigned char *p) {
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)(p)));
}
__device__ __forceinline__ u32x2 read_tr8(const unsigned char *p) {
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr8_b64_v2i32((__attribute__((address_space(3))) i32x2 *)(p)));
}

// A fragment of values in three parts, for tiles in which some row does not see some
// key: the finite numbers, and ones where an infinity pulls up or down (a NaN does
// both).  The first meets the probabilities; the others meet ones and zeros, for
// seen and not, and only say where a row sees such a value.
template <typename X> struct Parts {
    typedef X x8 __attribute__((ext_vector_type(8)));
    x8 finite, up, down;
    __device__ __forceinline__ explicit Parts(u32x4 v) {
        typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));
        constexpr uint16_t kExp = std::is_same_v<X, _Float16> ? 0x7C00 : 0x7F80;
        const u16x8 h = __builtin_bit_cast(u16x8, v);
        u16x8 f, u, d;
        const uint16_t one = __builtin_bit_cast(uint16_t, (X)1.f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool bad = (h[i] & kExp) == kExp;
            f[i] = bad ? (uint16_t)0 : h[i];
            u[i] = bad && h[i] != (0x8000 | kExp) ? one : (uint16_t)0;
            d[i] = bad && h[i] != kExp ? one : (uint16_t)0;
        }
        finite = __builtin_bit_cast(x8, f), up = __builtin_bit_cast(x8, u), down = __builtin_bit_cast(x8, d);
    }
};

// A key's scale: under an infinite one its elements are infinities of both signs, or NaN
// where the code is 0, and so its score is NaN, not the infinity that scaling the sum gives.
__device__ __forceinline__ float finite_or_nan(float s) { return __builtin_isfinite(s) ? s : NAN; }

// How the value scales of a tile of keys enter, one key a lane; the same for all lanes.
constexpr float kUneven = 1024.f;  // in place of the exponent
struct ValueUnit {
    int exp = 0;  // biased exponent of a power of two above the scales of the last even tile
    // `bits` of the magnitude of the lane's scale; `counts` where its key is in the cache and the scale finite.
    // Returns the exponent of the power by which the tile's scales are to be divided, or kUneven where they stay
    // as they are.
    __device__ __forceinline__ float of_tile(uint32_t bits, bool counts) {
        const int e = (int)(bits >> 23);
        if (__any(counts && (e >= exp || e < exp - 7))) {
            int most = counts ? e : 0, least = counts ? e : 255;
#pragma unroll
            for (int x = 1; x < 64; x *= 2) {
                most = max(most, __shfl_xor(most, x, 64));
                least = min(least, __shfl_xor(least, x, 64));
            }
            most = __builtin_amdgcn_readfirstlane(most), least = __builtin_amdgcn_readfirstlane(least);
            if (most - least > 6) return kUneven;
            exp = most + 1;
        }
        return (float)(exp - 127);
    }
};
__device__ __forceinline__ float in_unit(float scale, float unit) {
    return unit == kUneven ? scale : __builtin_amdgcn_ldexpf(scale, -(int)unit);
}
// A row's exponents, before it has seen anything: below all others, and yet a number.
constexpr float kNoExponent = -3.4028235e38f;
// mo after a tile whose largest product has the exponent u.
__device__ __forceinline__ float product_exponent(float mo, float u) { return u > mo + (kSlack + kLift) ? u - kLift : mo; }
// The exponent that an even tile's probabilities are taken relative to (an uneven one's: m).  Where it is kFar above m the
// products are nothing in fp16 (below 2^-52), while the sum still gets what the row sees.
constexpr float kFar = 60.f;
__device__ __forceinline__ float tile_exponent(float m, float mo, float unit) {
    return fminf(mo - unit, m + kFar);
}
// An uneven tile's scale for a row: the product with the probability 2^(x - m) is in the row's unit.
__device__ __forceinline__ float uneven_scale(float scale, float m, float mo) {
    const float v = scale * fminf(__builtin_amdgcn_exp2f(m - mo), 0x1p126f);
    return __builtin_isinf(v) && __builtin_isfinite(scale) ? copysignf(0x1p126f, scale) : v;
}
// An output and its sum: zeros where no key was seen.
__device__ __forceinline__ float divide(float o, float l) { return l > 0.f || l != l ? o / l : 0.f; }
#endif

}  // namespace cbs
