// k_int8_linear.hip -- the product of the linear layer in 8-bit integers and its
// epilogue: y[m][n] = act((sum_k a[m][k] w[n][k]) * sa[m] * sw[n] + bias[n]).
//
// Two kernels.  `linear_stream` is for few rows of x, where the layer is a read
// of w: every wave takes the fragments of w straight from memory into the matrix
// instruction, with no shared memory between, and the waves of a workgroup
// divide K.  `linear_tile` is for many rows, where the matrix pipe is the
// bound: tiles of both operands go through LDS.  The sums are 32-bit integers and
// so the same whatever the order.
#include <hip/hip_runtime.h>

#include "b8_device.h"
#include "b8_linear.h"

namespace cbs {
namespace {

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

// --- few rows --------------------------------------------------------------------

constexpr int kStreamWaves = 8;
constexpr int kStreamThreads = 64 * kStreamWaves;
constexpr int kFusedBytes = 32768;  // codes of the fused form, in LDS

struct StreamParams {
    CodesLayout l;
    const int8_t *w;
    const float *w_scale, *bias;
    const void *x;
    int64_t x_stride;
    void *y;
    int M, N, K, dtype, act;
};

template <typename T>
__device__ __forceinline__ void store_act(void *y, int64_t at, int sum, float sa, float sw, float bias, int act) {
    Value<T>::store1((T *)y + at, act == CBS_ACT_SILU ? linear_epilogue<T, true>(sum, sa, sw, bias)
                                                      : linear_epilogue<T, false>(sum, sa, sw, bias));
}

// One workgroup: 16 MT rows of x by 16 NT rows of w.  A step is 128 of K: two
// fragments (16 rows by 64) of each 16 rows.  Wave i takes the steps i, i + 8, ...,
// so that the workgroup reads 1 KiB of each row of w at a time, and holds
// one step's fragments while the next one's are on their way.
// w may start at any byte, and its rows with it.  The codes past K are zero, so
// what of w meets them does not matter; it is read inside w.
//
// ROWS > 0 (then M <= ROWS, MT = 1): the workgroup quantises x by itself, into
// LDS, with 8 / ROWS waves to a row, while its first fragments of w arrive.  It
// saves the launch and the pass before this one.
template <typename T, int MT, int NT, int ROWS>
__global__ __launch_bounds__(kStreamThreads) void linear_stream(const StreamParams p) {
    extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
    __shared__ float row_scales[ROWS > 0 ? ROWS : 1];
    __shared__ uint32_t row_tops[kStreamWaves];
    const int lane = (int)threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / 64);
    const int row = lane % 16, group = lane / 16;
    const int n0 = (int)blockIdx.x * 16 * NT, m0 = (int)blockIdx.y * 16 * MT;
    const int steps = p.l.Kp / 128, full = p.K / 128;  // the last step may be partial
    const int64_t size = (int64_t)p.N * p.K;
    const int8_t *wr[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) wr[j] = p.w + (int64_t)min(n0 + 16 * j + row, p.N - 1) * p.K + 16 * group;
    const int8_t *ar[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
        ar[i] = ROWS > 0 ? (const int8_t *)nullptr
                         : p.l.codes + (int64_t)min(m0 + 16 * i + row, p.l.rows - 1) * 64 + 16 * group;
    const int lds_row = min(row, p.M - 1) * 64 + 16 * group;

    i32x4 wf[2][NT][2], af[2][MT][2];
    auto load_w = [&](int s, i32x4(&f)[NT][2]) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int8_t *at = wr[j] + s * 128 + h * 64;
                f[j][h] = s < full ? __builtin_bit_cast(i32x4, ((const Any16 *)at)->v) : load_end(p.w, at - p.w, size);
            }
    };
    auto load_a = [&](int s, i32x4(&f)[MT][2]) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if constexpr (ROWS > 0) f[i][h] = *(const i32x4 *)(lds + (2 * s + h) * (ROWS * 64) + lds_row);
                else f[i][h] = *(const i32x4 *)(ar[i] + (int64_t)(2 * s + h) * p.l.rows * 64);
            }
    };

    if (wave < steps) load_w(wave, wf[0]);
    if constexpr (ROWS > 0) {
        constexpr int kTeam = kStreamThreads / ROWS;  // lanes to a row
        const int m = (int)threadIdx.x / kTeam, t = (int)threadIdx.x % kTeam;
        const T *x = (const T *)p.x + (int64_t)min(m, p.M - 1) * p.x_stride;
        auto chunk = [&](int k) {
            if (k + 8 <= p.K) return Value<T>::load8(x + k);
            f32x8 v = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (k + i < p.K) v[i] = Value<T>::load1(x + k + i);
            return v;
        };
        uint32_t top = 0;
        for (int k = t * 8; k < p.K; k += kTeam * 8) {
            const f32x8 v = chunk(k);
#pragma unroll
            for (int i = 0; i < 8; ++i) top = max(top, magnitude(v[i]));
        }
#pragma unroll
        for (int o = 1; o < 64; o *= 2) top = max(top, (uint32_t)__shfl_xor((int)top, o, 64));
        if (lane == 0) row_tops[wave] = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kTeam / 64; ++i) top = max(top, row_tops[m * (kTeam / 64) + i]);
        const float s = row_scale(top), inv = row_inverse(s, top);
        if (m < p.M) {
            for (int k = t * 8; k < p.l.Kp; k += kTeam * 8) {
                int c[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                if (inv != 0.f) row_codes8(chunk(k), s, inv, c);
                *(u32x2 *)(lds + (k >> 6) * (ROWS * 64) + m * 64 + (k & 63)) =
                    u32x2{pack_codes(c[0], c[1], c[2], c[3]), pack_codes(c[4], c[5], c[6], c[7])};
            }
            if (t == 0) row_scales[m] = s;
        }
        __syncthreads();
    }

    i32x4 acc[MT][NT] = {};
    auto product = [&](const i32x4(&a)[MT][2], const i32x4(&w)[NT][2]) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[i][h], w[j][h], acc[i][j], 0, 0, 0);
    };
    if (wave < steps) load_a(wave, af[0]);
    for (int s = wave; s < steps; s += 2 * kStreamWaves) {
        const int s1 = s + kStreamWaves, s2 = s + 2 * kStreamWaves;
        if (s1 < steps) {
            load_w(s1, wf[1]);
            load_a(s1, af[1]);
        }
        product(af[0], wf[0]);
        if (s1 < steps) {
            if (s2 < steps) {
                load_w(s2, wf[0]);
                load_a(s2, af[0]);
            }
            product(af[1], wf[1]);
        }
    }

    // the waves' sums meet in LDS; the codes there are no longer needed
    if constexpr (ROWS > 0) __syncthreads();
    int *part = (int *)lds;  // [wave][m][n]
    constexpr int kRow = 16 * NT, kOut = 16 * MT * kRow;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                part[wave * kOut + (16 * i + 4 * group + r) * kRow + 16 * j + row] = acc[i][j][r];
    __syncthreads();
    for (int e = (int)threadIdx.x; e < kOut; e += kStreamThreads) {
        const int m = m0 + e / kRow, n = n0 + e % kRow;
        if (m >= p.M || n >= p.N) continue;
        int sum = 0;
#pragma unroll
        for (int v = 0; v < kStreamWaves; ++v) sum += part[v * kOut + e];
        const float sa = ROWS > 0 ? row_scales[ROWS > 0 ? m : 0] : p.l.scales[m];
        const float sw = p.w_scale[n], bias = p.bias ? p.bias[n] : 0.f;
        const int64_t at = (int64_t)m * p.N + n;
        switch (p.dtype) {
            case CBS_DTYPE_F32: store_act<float>(p.y, at, sum, sa, sw, bias, p.act); break;
            case CBS_DTYPE_BF16: store_act<__bf16>(p.y, at, sum, sa, sw, bias, p.act); break;
            default: store_act<_Float16>(p.y, at, sum, sa, sw, bias, p.act);
        }
    }
}

// --- many rows -------------------------------------------------------------------

// Places a workgroup's tile so that the tiles of one XCD (workgroups go to the
// eight in turn) lie together: each takes a run of the tiles, in bands of 8 rows of tiles, and
// its L2 serves a patch of rows and columns.
struct Tile {
    int m, n;
};
__device__ __forceinline__ Tile place(int id, int m_tiles, int n_tiles) {
    const int total = m_tiles * n_tiles, xcd = id % 8, each = total / 8, more = total % 8;
    const int t = xcd * each + min(xcd, more) + id / 8;
    const int band = t / (8 * n_tiles), rows = min(8, m_tiles - 8 * band), in = t - band * 8 * n_tiles;
    return Tile{8 * band + in % rows, in / rows};
}

struct TileParams {
    CodesLayout l;
    const int8_t *w;
    int w_stride;
    const float *w_scale, *bias;
    void *y;
    int M, N, m_tiles, n_tiles;
};

typedef __attribute__((address_space(3))) void lds_void;

// BM x BN outputs, a wave 32 MB x 64 of them on v_mfma_i32_32x32x32_i8; K in
// steps of 128 through LDS, where loads write directly, one step ahead.
//
// An LDS row is 128 bytes of one row of an operand; its 16-byte pieces are
// exchanged by (row / 2) % 8, so that the 16 rows that a quarter of a wave reads
// at one k cover all banks.  The loads, which fill LDS in lane order, fetch the
// pieces in that order from memory, through buffers that end with the operand's
// part: rows past it come as zero.
template <typename T, bool SILU, int BM, int BN, int MB>
__global__ __launch_bounds__(64 * (BM / (32 * MB)) * (BN / 64), 2) void linear_tile(const TileParams p) {
    constexpr int kWavesN = BN / 64, kWaves = BM / (32 * MB) * kWavesN, NB = 2;
    constexpr int kLoadsA = BM / 8 / kWaves, kLoadsB = BN / 8 / kWaves;  // of 8 rows, a wave and step
    __shared__ __attribute__((aligned(16))) int8_t a0[BM * 128], b0[BN * 128], a1[BM * 128], b1[BN * 128];
    const int lane = (int)threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / 64);
    const Tile t = place((int)blockIdx.x, p.m_tiles, p.n_tiles);
    const int m0 = t.m * BM, n0 = t.n * BN;

    // staging: lane i of a load fetches the piece that belongs at i % 8 of row i / 8
    const uint32_t block = (uint32_t)p.l.rows * 64;
    uint32_t off_a[kLoadsA], off_b[kLoadsB];
#pragma unroll
    for (int i = 0; i < kLoadsA; ++i) {
        const int r = (wave * kLoadsA + i) * 8 + lane / 8, c = (lane % 8) ^ ((r >> 1) & 7);
        off_a[i] = c / 4 * block + (uint32_t)(r * 64 + c % 4 * 16);
    }
#pragma unroll
    for (int i = 0; i < kLoadsB; ++i) {
        const int r = (wave * kLoadsB + i) * 8 + lane / 8, c = (lane % 8) ^ ((r >> 1) & 7);
        off_b[i] = (uint32_t)(r * p.w_stride + c * 16);
    }
    const int8_t *base_a = p.l.codes + (int64_t)m0 * 64, *base_b = p.w + (int64_t)n0 * p.w_stride;
    const uint32_t size_a = 2 * block - (uint32_t)m0 * 64, size_b = (uint32_t)(min(BN, p.N - n0) * p.w_stride);
    auto stage = [&](int s, int8_t *a, int8_t *b) {
        const auto ra = make_rsrc(base_a + (int64_t)s * 2 * block, size_a);
        const auto rb = make_rsrc(base_b + s * 128, size_b - (uint32_t)s * 128);
#pragma unroll
        for (int i = 0; i < kLoadsA; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void *)(a + (wave * kLoadsA + i) * 1024), 16, (int)off_a[i],
                                                     0, 0, 0);
#pragma unroll
        for (int i = 0; i < kLoadsB; ++i)  // past K: the next row or zero, against codes of zero
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void *)(b + (wave * kLoadsB + i) * 1024), 16, (int)off_b[i],
                                                     0, 0, 0);
    };

    const int wm = wave / kWavesN * 32 * MB, wn = wave % kWavesN * 64, r32 = lane % 32, half = lane / 32;
    const int swap = (r32 >> 1) & 7;  // the same for every 32 rows
    i32x16 acc[MB][NB] = {};
    auto compute = [&](const int8_t *a, const int8_t *b) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int at = ((2 * k + half) ^ swap) * 16 + r32 * 128;
            i32x4 af[MB], bf[NB];
#pragma unroll
            for (int j = 0; j < NB; ++j) bf[j] = *(const i32x4 *)(b + (wn + 32 * j) * 128 + at);
#pragma unroll
            for (int i = 0; i < MB; ++i) af[i] = *(const i32x4 *)(a + (wm + 32 * i) * 128 + at);
#pragma unroll
            for (int i = 0; i < MB; ++i)
#pragma unroll
                for (int j = 0; j < NB; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(af[i], bf[j], acc[i][j], 0, 0, 0);
        }
    };
    const int steps = p.l.Kp / 128;
    stage(0, a0, b0);
    int s = 0;
    for (; s + 2 < steps; s += 2) {
        __syncthreads();  // this step's tiles are there, the other pair is free
        stage(s + 1, a1, b1);
        compute(a0, b0);
        __syncthreads();
        stage(s + 2, a0, b0);
        compute(a1, b1);
    }
    __syncthreads();
    if (s + 1 < steps) stage(s + 1, a1, b1);
    compute(a0, b0);
    __syncthreads();
    if (s + 1 < steps) {
        compute(a1, b1);
        __syncthreads();
    }

    // A lane holds one n and, of every 32 rows, 16.  32 rows at a time go through
    // the wave's own part of LDS (64 sums and a pad a row), so that a lane then
    // has 8 neighbouring n and a store covers whole lines.
    constexpr int kPitch = 68;  // sums a row
    constexpr int kEach = kWaves / 4;
    static_assert(kWaves % 4 == 0 && BM == BN && 32 * kPitch * 4 * kEach <= 128 * BM, "a quarter of the waves to each array");
    int *tile = (int *)(wave / kEach == 0 ? a0 : wave / kEach == 1 ? b0 : wave / kEach == 2 ? a1 : b1) +
                wave % kEach * (32 * kPitch);
    const int n = n0 + wn + lane % 8 * 8;
    float sw[8], bias[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        sw[e] = p.w_scale[min(n + e, p.N - 1)];
        bias[e] = p.bias ? p.bias[min(n + e, p.N - 1)] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < MB; ++i) {
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                tile[(8 * (r / 4) + 4 * half + r % 4) * kPitch + 32 * j + r32] = acc[i][j][r];
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int row = 8 * q + lane / 8, m = m0 + wm + 32 * i + row;
            const i32x4 *from = (const i32x4 *)(tile + row * kPitch + lane % 8 * 8);
            const i32x4 lo = from[0], hi = from[1];
            if (m >= p.M) continue;
            const float sa = p.l.scales[m];
            f32x8 v;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = linear_epilogue<T, SILU>(e < 4 ? lo[e % 4] : hi[e % 4], sa, sw[e], bias[e]);
            T *to = (T *)p.y + (int64_t)m * p.N + n;
            if (n + 8 <= p.N) {
                Value<T>::store8(to, v);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (n + e < p.N) Value<T>::store1(to + e, v[e]);
            }
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// Rows of w at any byte to rows of Kp, each at a multiple of 16, for the tile kernel's
// loads.
__global__ __launch_bounds__(256) void align_rows(const int8_t *__restrict__ w, int8_t *__restrict__ to, int N, int K,
                                                  int Kp) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int each = Kp / 16;
    const int64_t n = i / each;
    if (n >= N) return;
    const int k = (int)(i - n * each) * 16;
    *(i32x4 *)(to + n * Kp + k) = load_end(w, n * K + k, (int64_t)N * K);
}

// --- choice ----------------------------------------------------------------------

enum Kind { kStream, kTile128, kTile256 };
// By the number of tiles that a kernel makes of the output, against the 256 CUs.
Kind kind_of(int64_t M, int64_t N) {
    const int64_t t256 = ((M + 255) / 256) * ((N + 255) / 256), t128 = ((M + 127) / 128) * ((N + 127) / 128);
    if (M <= 64) return kStream;
    if (t256 >= 192) return kTile256;
    return t128 >= 128 ? kTile128 : kStream;
}
bool needs_copy(int64_t M, int64_t N, int64_t K) { return K % 16 != 0 && kind_of(M, N) != kStream; }

template <typename T, int MT, int NT, int ROWS> hipError_t launch_stream4(const StreamParams &p, hipStream_t st) {
    const dim3 grid((p.N + 16 * NT - 1) / (16 * NT), (p.M + 16 * MT - 1) / (16 * MT));
    const size_t sums = (size_t)kStreamWaves * 16 * MT * 16 * NT * 4, codes = (size_t)ROWS * p.l.Kp;
    linear_stream<T, MT, NT, ROWS><<<grid, kStreamThreads, sums > codes ? sums : codes, st>>>(p);
    return hipGetLastError();
}
template <typename T, int MT, int ROWS> hipError_t launch_stream3(const StreamParams &p, hipStream_t st) {
    // 32 rows of w to a workgroup where that leaves two for every CU, else 16
    const bool two = (int64_t)((p.N + 31) / 32) * ((p.M + 16 * MT - 1) / (16 * MT)) >= 512;
    return two ? launch_stream4<T, MT, 2, ROWS>(p, st) : launch_stream4<T, MT, 1, ROWS>(p, st);
}
template <typename T> hipError_t launch_stream(const LinearArgs &a, const CodesLayout &l, hipStream_t st) {
    const StreamParams p{l, a.w, a.w_scale, a.bias, a.x, a.x_stride, a.y, a.M, a.N, a.K, a.dtype, a.act};
    if (a.M <= 1 && (int64_t)l.Kp <= kFusedBytes) return launch_stream3<T, 1, 1>(p, st);
    if (a.M <= 2 && (int64_t)l.Kp * 2 <= kFusedBytes) return launch_stream3<T, 1, 2>(p, st);
    if (a.M <= 4 && (int64_t)l.Kp * 4 <= kFusedBytes) return launch_stream3<T, 1, 4>(p, st);
    const hipError_t e = launch_quant_rows(a, l, st);
    if (e != hipSuccess) return e;
    // from here on x is not read: one type of the kernel serves all
    if (a.M <= 16) return launch_stream3<float, 1, 0>(p, st);
    if (a.M <= 32) return launch_stream3<float, 2, 0>(p, st);
    if (a.M <= 48) return launch_stream3<float, 3, 0>(p, st);
    return launch_stream3<float, 4, 0>(p, st);
}

template <typename T, bool SILU> hipError_t launch2(const LinearArgs &a, const CodesLayout &l, hipStream_t st) {
    const Kind kind = kind_of(a.M, a.N);
    const bool copy = needs_copy(a.M, a.N, a.K);
    // where only w's start is off 16 bytes there is no room for a copy
    if (kind == kStream || (!copy && (uintptr_t)a.w % 16 != 0)) return launch_stream<T>(a, l, st);
    hipError_t e = launch_quant_rows(a, l, st);
    if (e != hipSuccess) return e;
    TileParams p{l, a.w, a.K, a.w_scale, a.bias, a.y, a.M, a.N, 0, 0};
    if (copy) {
        int8_t *to = l.codes + (int64_t)l.rows * l.Kp;
        align_rows<<<(unsigned)(((int64_t)a.N * (l.Kp / 16) + 255) / 256), 256, 0, st>>>(a.w, to, a.N, a.K, l.Kp);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        p.w = to, p.w_stride = l.Kp;
    }
    const int b = kind == kTile256 ? 256 : 128;
    p.m_tiles = (a.M + b - 1) / b, p.n_tiles = (a.N + b - 1) / b;
    const unsigned grid = (unsigned)(p.m_tiles * p.n_tiles);
    if (kind == kTile256) linear_tile<T, SILU, 256, 256, 4><<<grid, 512, 0, st>>>(p);
    else linear_tile<T, SILU, 128, 128, 2><<<grid, 256, 0, st>>>(p);
    return hipGetLastError();
}
template <typename T> hipError_t launch1(const LinearArgs &a, const CodesLayout &l, hipStream_t st) {
    return a.act == CBS_ACT_SILU ? launch2<T, true>(a, l, st) : launch2<T, false>(a, l, st);
}

}  // namespace

int64_t linear_workspace(int64_t M, int64_t N, int64_t K) {
    const CodesLayout l = codes_layout(nullptr, M, K);
    return l.bytes + (needs_copy(M, N, K) ? N * l.Kp : 0);
}

hipError_t launch_int8_linear(const LinearArgs &a, int num_cu, hipStream_t st) {
    (void)num_cu;
    const CodesLayout l = codes_layout(a.workspace, a.M, a.K);
    switch (a.dtype) {
        case CBS_DTYPE_F32: return launch1<float>(a, l, st);
        case CBS_DTYPE_BF16: return launch1<__bf16>(a, l, st);
        default: return launch1<_Float16>(a, l, st);
    }
}

}  // namespace cbs
