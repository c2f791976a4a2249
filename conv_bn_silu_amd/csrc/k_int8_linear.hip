// k_int8_linear.hip -- the product of the linear layer in 8-bit integers and its
// epilogue: y[m][n] = act((sum_k a[m][k] w[n][k]) * sa[m] * sw[n] + bias[n]).
//
// Three kernels.  `linear_stream` is for few tiles of output, where the layer is a
// read of w: every wave takes the fragments of w straight from memory into the
// matrix instruction, with no shared memory between, and the waves of a workgroup
// divide K.  In `linear_ring` tiles of both operands go through LDS, with loads four steps
// ahead, and `linear_tile` is the same for outputs that fill the CUs, where the matrix
// pipe is the bound.  The sums are 32-bit integers and so the same whatever the order; where
// few tiles have long sums, several workgroups of linear_ring divide a tile's K.
//
// Measured, us a call with the pass that quantises x (copying at 6.3 TB/s, matrix
// products at 2.1 POP/s would take the second figure):
//   1 x 4096 x 4096      stream     6.6   2.7      256 x 4096 x 4096     ring 64    18   4.1
//   1 x 16384 x 4096     stream    15.3  10.7      1024 x 4096 x 4096    ring 128   33    16
//   40 x 16384 x 4096    ring 64   18.7  10.9      4096 x 4096 x 4096    tile       81    65
//   128 x 16384 x 4096   ring 64   22.9  11.5      8192 x 8192 x 8192    tile      529   524
//   128 x 1024 x 8192    4 parts   17.3   1.7
// The pass over x takes 4 us of it for few rows, 5 to 8 for 256 to 1024 and 47 for 8192 x 8192.
// Rows that come in 8 bits spare it: a norm (add_rms_norm) and the layer, us, with the values in 16 bits between them and with
// the rows in 8: 1 x 4096 x 4096 11.0 and 10.8, 16 x 4096 x 4096 14.8 and 11.0, 1024 x 4096 x 4096 39 and 35,
// 8192 x 8192 x 8192 590 and 581.
// 1024 x 4096 x 4096 has 256 tiles of 128, one to a CU: 25 us for 32 steps with four waves to feed a CU's matrix
// pipes, where 256-tiles (64 of them) would leave three CUs of four idle.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "b8_device.h"
#include "b8_linear.h"

namespace cbs {
namespace {

// --- few rows --------------------------------------------------------------------

constexpr int kStreamWaves = 8;
constexpr int kStreamThreads = 64 * kStreamWaves;
// The fused form of linear_stream: most rows, and most codes in LDS.  4096 x 4096, fused and
// not: 4 rows 8.5 and 9.1 us, 8 rows 11.0 and 9.2.
constexpr int kFusedRows = 16, kFusedBytes = 16384;

struct StreamParams {
    CodesLayout l;
    const int8_t *w;
    const float *w_scale, *bias;
    const void *x;
    int64_t x_stride;
    void *y;
    int M, N, K, dtype, act;
    int m_tile;  // tile of rows of x that the launch begins with
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
    const int n0 = (int)blockIdx.x * 16 * NT, m0 = ((int)blockIdx.y + p.m_tile) * 16 * MT;
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
        for (int o = 1; o < (kTeam < 64 ? kTeam : 64); o *= 2) top = max(top, (uint32_t)__shfl_xor((int)top, o, 64));
        if constexpr (kTeam > 64) {
            if (lane == 0) row_tops[wave] = top;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kTeam / 64; ++i) top = max(top, row_tops[m * (kTeam / 64) + i]);
        }
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
    // linear_ring, K divided between `splits` workgroups: their sums, [split][tile][wave][32][64] in
    // the order of the registers, and how many of a tile's are there
    int splits, split_steps;
    int *sums, *arrived;
};

// Stores a wave's sums, 32 MB x 64 of them from (m0, n0).  A lane holds one n and, of every
// 32 rows, 16.  32 rows at a time go through the wave's own part of LDS (64 sums
// and a pad a row), so that a lane then has 8 neighbouring n and a store covers
// whole lines.
constexpr int kTilePitch = 68, kTileBytes = 32 * kTilePitch * 4;
template <typename T, bool SILU, int MB>
__device__ __forceinline__ void store_sums(const TileParams &p, const i32x16 (&acc)[MB][2], int *tile, int m0, int n0) {
    const int lane = (int)threadIdx.x % 64, r32 = lane % 32, half = lane / 32;
    const int n = n0 + lane % 8 * 8;
    float sw[8], bias[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        sw[e] = p.w_scale[min(n + e, p.N - 1)];
        bias[e] = p.bias ? p.bias[min(n + e, p.N - 1)] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < MB; ++i) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                tile[(8 * (r / 4) + 4 * half + r % 4) * kTilePitch + 32 * j + r32] = acc[i][j][r];
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int row = 8 * q + lane / 8, m = m0 + 32 * i + row;
            const i32x4 *from = (const i32x4 *)(tile + row * kTilePitch + lane % 8 * 8);
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

typedef __attribute__((address_space(3))) void lds_void;

// A step's products of a wave, from its rows of the two operands in LDS.  The fragments
// of AHEAD of the step's four parts are on their way at a time, and `issue` (a quarter of a
// later step's loads) goes between the parts; the order is held.  Left alone the compiler
// reads a part when it is wanted, and the matrix pipe waits for each; and loads issued all
// at once hold the wave up for as long as the CU takes to serve them (64 bytes a
// clock: half of a step).
template <int MB, int AHEAD, typename F>
__device__ __forceinline__ void multiply(i32x16 (&acc)[MB][2], const int8_t *a, const int8_t *b, int half, int swap,
                                         F &&issue) {
    i32x4 af[AHEAD][MB], bf[AHEAD][2];
    auto read = [&](int k) {
        const int at = ((2 * k + half) ^ swap) * 16;
#pragma unroll
        for (int j = 0; j < 2; ++j) bf[k % AHEAD][j] = *(const i32x4 *)(b + 32 * j * 128 + at);
#pragma unroll
        for (int i = 0; i < MB; ++i) af[k % AHEAD][i] = *(const i32x4 *)(a + 32 * i * 128 + at);
    };
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) read(k);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        __builtin_amdgcn_sched_barrier(0);
        issue(k);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(af[k % AHEAD][i], bf[k % AHEAD][j], acc[i][j], 0, 0, 0);
        if (k + AHEAD < 4) {
            __builtin_amdgcn_sched_barrier(0);
            read(k + AHEAD);
        }
    }
}

// Where a wave's loads of an operand's step come from and go: load i fills 8 rows of 128
// bytes; lane j of it fetches the piece that belongs at j % 8 of row j / 8.
//
// An LDS row's 16-byte pieces are exchanged by (row / 2) % 8, so that the 16 rows that a
// quarter of a wave reads at one k cover all banks.  The loads, which fill LDS in lane
// order, fetch the pieces in that order from memory, through buffers that end with the
// operand's part: rows past it come as zero, and a buffer of no bytes is a step past
// the last.
constexpr int kLoads = 4;  // of each operand, a wave and step
struct Loads {
    const int8_t *base_a, *base_b;
    uint32_t off_a[kLoads], off_b[kLoads], size_a, size_b;
    int64_t step_a;
    int wave, steps;
    // The steps [s0, s0 + n) of K.
    __device__ __forceinline__ Loads(const TileParams &p, int m0, int n0, int bn, int w, int lane, int s0, int n) {
        const uint32_t block = (uint32_t)p.l.rows * 64;
        wave = w, steps = n;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int r = (wave * kLoads + i) * 8 + lane / 8, c = (lane % 8) ^ ((r >> 1) & 7);
            off_a[i] = c / 4 * block + (uint32_t)(r * 64 + c % 4 * 16);
        }
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int r = (wave * kLoads + i) * 8 + lane / 8, c = (lane % 8) ^ ((r >> 1) & 7);
            off_b[i] = (uint32_t)(r * p.w_stride + c * 16);
        }
        step_a = 2 * (int64_t)block;
        base_a = p.l.codes + (int64_t)m0 * 64 + s0 * step_a, base_b = p.w + (int64_t)n0 * p.w_stride + s0 * 128;
        size_a = 2 * block - (uint32_t)m0 * 64, size_b = (uint32_t)(min(bn, p.N - n0) * p.w_stride) - (uint32_t)s0 * 128;
    }
    // A step's part of the operands, and its size.
    __device__ __forceinline__ const int8_t *a_at(int s) const { return base_a + s * step_a; }
    __device__ __forceinline__ const int8_t *b_at(int s) const { return base_b + s * 128; }
    __device__ __forceinline__ uint32_t a_bytes(int s) const { return __builtin_amdgcn_readfirstlane(s < steps ? size_a : 0); }
    __device__ __forceinline__ uint32_t b_bytes(int s) const {
        return __builtin_amdgcn_readfirstlane(s < steps ? size_b - (uint32_t)s * 128 : 0);
    }
};

// BM x BN outputs, a wave 32 MB x 64 of them on v_mfma_i32_32x32x32_i8; K in
// steps of 128 through LDS, where loads write directly, one step ahead.
template <typename T, bool SILU, int BM, int BN, int MB>
__global__ __launch_bounds__(64 * (BM / (32 * MB)) * (BN / 64), 2) void linear_tile(const TileParams p) {
    constexpr int kWavesN = BN / 64, kWaves = BM / (32 * MB) * kWavesN;
    static_assert(BM == BN && BM / 8 / kWaves == kLoads, "");
    __shared__ __attribute__((aligned(16))) int8_t a0[BM * 128], b0[BN * 128], a1[BM * 128], b1[BN * 128];
    const int lane = (int)threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / 64);
    const Tile t = place((int)blockIdx.x, p.m_tiles, p.n_tiles);
    const int m0 = t.m * BM, n0 = t.n * BN;
    const Loads loads(p, m0, n0, BN, wave, lane, 0, p.l.Kp / 128);
    const int wm = wave / kWavesN * 32 * MB, wn = wave % kWavesN * 64, r32 = lane % 32, half = lane / 32;
    const int swap = (r32 >> 1) & 7;  // the same for every 32 rows
    const int at_a = (wm + r32) * 128, at_b = (wn + r32) * 128;
    i32x16 acc[MB][2] = {};
    // Load i of either operand of step s.  Past K the next row of w or zero comes, against codes of zero.
    auto issue = [&](int s, int i, int8_t *a, int8_t *b) {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(loads.a_at(s), loads.a_bytes(s)), (lds_void *)(a + (wave * kLoads + i) * 1024), 16,
                                                 (int)loads.off_a[i], 0, 0, 0);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(loads.b_at(s), loads.b_bytes(s)), (lds_void *)(b + (wave * kLoads + i) * 1024), 16,
                                                 (int)loads.off_b[i], 0, 0, 0);
    };
#pragma unroll
    for (int i = 0; i < kLoads; ++i) issue(0, i, a0, b0);
    for (int s = 0; s < loads.steps; s += 2) {
        __syncthreads();  // this step's tiles are there, the other pair is free
        multiply<MB, 2>(acc, a0 + at_a, b0 + at_b, half, swap, [&](int k) { issue(s + 1, k, a1, b1); });
        __syncthreads();
        if (s + 1 < loads.steps)
            multiply<MB, 2>(acc, a1 + at_a, b1 + at_b, half, swap, [&](int k) { issue(s + 2, k, a0, b0); });
    }
    __syncthreads();
    constexpr int kEach = kWaves / 4;
    static_assert(kWaves % 4 == 0 && kTileBytes * kEach <= 128 * BM, "a quarter of the waves to each array");
    int8_t *const mine = wave / kEach == 0 ? a0 : wave / kEach == 1 ? b0 : wave / kEach == 2 ? a1 : b1;
    store_sums<T, SILU, MB>(p, acc, (int *)(mine + wave % kEach * kTileBytes), m0 + wm, n0 + wn);
}

// A workgroup of linear_ring has the sums over its part of K.  True in the one of a tile's that
// ends last, which then has all of them: the others' sums are in memory and it adds them.
// Sums are written through to where every XCD sees them and read from there: fences, which
// write back and empty an L2, took 50 us and more in all.
__device__ __forceinline__ bool last_of_tile(const TileParams &p, i32x16 (&acc)[1][2], int id, int split, int wave, int lane) {
    __shared__ int before;
    const int all = p.m_tiles * p.n_tiles;
    auto at = [&](int s) { return (uint64_t *)p.sums + ((int64_t)(s * all + id) * 2 + wave) * 1024 + lane; };
    uint64_t *const mine = at(split);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int r = 0; r < 8; ++r)
            __hip_atomic_store(mine + (8 * j + r) * 64, (uint64_t)(uint32_t)acc[0][j][2 * r + 1] << 32 | (uint32_t)acc[0][j][2 * r],
                               __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __builtin_amdgcn_s_waitcnt(0);  // they have arrived
    asm volatile("" ::: "memory");
    __syncthreads();
    if (threadIdx.x == 0) before = __hip_atomic_fetch_add(p.arrived + id, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (before != p.splits - 1) return false;
    asm volatile("" ::: "memory");
    for (int s = 0; s < p.splits; ++s) {
        if (s == split) continue;
        const uint64_t *const from = at(s);
        uint64_t v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = __hip_atomic_load(from + i * 64, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            acc[0][i / 8][i % 8 * 2] += (int)(uint32_t)v[i];
            acc[0][i / 8][i % 8 * 2 + 1] += (int)(uint32_t)(v[i] >> 32);
        }
    }
    return true;
}

// The same for fewer tiles than keep every CU's matrix pipes fed: then a step is done long
// before the next one's loads arrive, so that here the loads run four steps ahead, in
// registers (which a wave has to spare), and pass into one of two LDS buffers a
// step ahead.
template <typename T, bool SILU, int BM, int BN, int MB>
__global__ __launch_bounds__(64 * (BM / (32 * MB)) * (BN / 64)) void linear_ring(const TileParams p) {
    constexpr int kWavesN = BN / 64, kWaves = BM / (32 * MB) * kWavesN;
    constexpr int kSets = 4;
    static_assert(BM == BN && BM / 8 / kWaves == kLoads, "");
    constexpr int kB = BM * 128;  // where a buffer's part of w begins
    __shared__ __attribute__((aligned(16))) int8_t lds[2][2 * kB];
    const int lane = (int)threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / 64);
    const int id = (int)blockIdx.x, split = MB == 1 ? (int)blockIdx.y : 0;
    const Tile t = place(id, p.m_tiles, p.n_tiles);
    const int m0 = t.m * BM, n0 = t.n * BN;
    const int steps = p.l.Kp / 128, s0 = MB == 1 ? split * p.split_steps : 0;
    const Loads loads(p, m0, n0, BN, wave, lane, s0, MB == 1 ? min(p.split_steps, steps - s0) : steps);
    const int wm = wave / kWavesN * 32 * MB, wn = wave % kWavesN * 64, r32 = lane % 32, half = lane / 32;
    const int swap = (r32 >> 1) & 7;
    i32x16 acc[MB][2] = {};
    u32x4 ra[kSets][kLoads], rb[kSets][kLoads];
    const int to = wave * kLoads * 1024 + lane * 16;
    auto fetch = [&](int s, int set, int i) {
        ra[set][i] = buf_load16(make_rsrc(loads.a_at(s), loads.a_bytes(s)), loads.off_a[i]);
        rb[set][i] = buf_load16(make_rsrc(loads.b_at(s), loads.b_bytes(s)), loads.off_b[i]);
    };
    auto pass = [&](int set, int i, int8_t *buf) {
        *(u32x4 *)(buf + to + i * 1024) = ra[set][i];
        *(u32x4 *)(buf + kB + to + i * 1024) = rb[set][i];
    };
    auto turn = [&](int s, auto turn_of_4) {
        constexpr int kNow = decltype(turn_of_4)::value, kNext = (kNow + 1) % kSets;
        const int8_t *const buf = lds[kNow % 2];
        // what this wave has written is there (lgkmcnt(0); loads go on), and so is what the others have
        __builtin_amdgcn_s_waitcnt(15 | 3 << 14 | 7 << 4);
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        multiply<MB, 2>(acc, buf + (wm + r32) * 128, buf + kB + (wn + r32) * 128, half, swap, [&](int k) {
            pass(kNext, k, lds[1 - kNow % 2]);
            fetch(s + 1 + kSets, kNext, k);
        });
    };
    // in this order: the waits in the loop count on it
#pragma unroll
    for (int set = 0; set < kSets; ++set)
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            fetch(set, set, i);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        pass(0, i, lds[0]);
        fetch(kSets, 0, i);
        __builtin_amdgcn_sched_barrier(0);
    }
    using std::integral_constant;
    int s = 0;
    for (; s + 4 <= loads.steps; s += 4) {  // without a way out in between, where the waits would have to be for the worst
        turn(s, integral_constant<int, 0>{});
        turn(s + 1, integral_constant<int, 1>{});
        turn(s + 2, integral_constant<int, 2>{});
        turn(s + 3, integral_constant<int, 3>{});
    }
    if (s < loads.steps) turn(s, integral_constant<int, 0>{});
    if (s + 1 < loads.steps) turn(s + 1, integral_constant<int, 1>{});
    if (s + 2 < loads.steps) turn(s + 2, integral_constant<int, 2>{});
    if constexpr (MB == 1)
        if (p.splits > 1 && !last_of_tile(p, acc, id, split, wave, lane)) return;
    __syncthreads();
    static_assert(kTileBytes * kWaves <= 4 * kB, "");
    store_sums<T, SILU, MB>(p, acc, (int *)(lds[0] + wave * kTileBytes), m0 + wm, n0 + wn);
}

// --- choice ----------------------------------------------------------------------

// By the number of tiles that a kernel makes of the output, against the CUs of the whole GPU: a constant,
// for the workspace, which depends on the choice, is asked for without a handle.  Where
// the choice changes, measured at K 2048 and 8192, in us (ring 64 with K whole; divided below):
//   M x N         linear_stream   ring 64       ring 128      tile 256
//   64 x 4096     10.0, 19.9      11.8, 24.2
//   96 x 4096     12.4, 28.3      12.2, 24.6
//   512 x 4096    29.4, 73.6      16.9, 35.1    19.5, 40.8
//   768 x 4096    40.4, 106       20.7, 47.8    20.5, 43.6
//   32 x 8192     10.9, 22.1      12.0, 23.2
//   32 x 16384    13.5, 37.9      12.9, 28.3
//   2048 x 8192   (K 4096)        117           86.3          70.4
constexpr int64_t kCus = 256;
enum Kind { kStream, kRing64, kRing128, kTile256 };
// Rows of the fused form for M rows of x, 0 where it does not serve them.
int fused_rows(int64_t M, int64_t K) {
    int rows = 1;
    while (rows < M) rows *= 2;
    return rows <= kFusedRows && rows * ((K + 127) / 128 * 128) <= kFusedBytes ? rows : 0;
}
int64_t tiles(int64_t M, int64_t N, int64_t b) { return ((M + b - 1) / b) * ((N + b - 1) / b); }
Kind kind_of(int64_t M, int64_t N, int64_t K) {
    if (fused_rows(M, K)) return kStream;
    // rows of w that start at odd bytes are read by linear_stream as they are, and have to be copied for the others
    if (K % 16 != 0 && M <= 128) return kStream;
    if (tiles(M, N, 256) >= kCus * 3 / 4) return kTile256;
    if (tiles(M, N, 128) >= kCus * 5 / 8) return kRing128;
    if (M > 32 && K > 6144) return kRing64;  // which divides K
    return tiles(M, N, 64) >= (M <= 32 ? kCus : kCus * 3 / 8) ? kRing64 : kStream;
}
// Workgroups of ring 64 that divide K: as many as leave one to a CU, with 16 steps for each, for
// bringing the sums together takes as long as about 16.  Whole and divided, us:
//   M x N         K 4096          K 8192        K 14336
//   64 x 1024     11.7, 13.1      18.7, 16.4    29.6, 21.5
//   96 x 4096     15.3, 14.1      24.0, 19.2    37.8, 27.4
//   512 x 1024    17.4, 16.3      26.0, 21.3    40.2, 29.7
//   256 x 4096    16.2, 17.7      24.7, 24.4    39.2, 36.5   (2 to a CU)
// (64 x 1024 whole is linear_stream.)
int splits_of(int64_t M, int64_t N, int64_t K) {
    if (kind_of(M, N, K) != kRing64) return 1;
    return (int)std::max<int64_t>(1, std::min<int64_t>(kCus / tiles(M, N, 64), (K + 127) / 128 / 16));
}
bool needs_copy(int64_t M, int64_t N, int64_t K) { return K % 16 != 0 && kind_of(M, N, K) != kStream; }

template <typename T, int MT, int NT, int ROWS> hipError_t launch_stream4(StreamParams p, hipStream_t st) {
    constexpr int kMost = 32768;  // tiles of rows to a launch: a grid's second dimension ends at 65535
    const int m_tiles = (p.M + 16 * MT - 1) / (16 * MT);
    const size_t sums = (size_t)kStreamWaves * 16 * MT * 16 * NT * 4, codes = (size_t)ROWS * p.l.Kp;
    hipError_t e = hipSuccess;
    for (; p.m_tile < m_tiles && e == hipSuccess; p.m_tile += kMost) {
        const dim3 grid((p.N + 16 * NT - 1) / (16 * NT), std::min(kMost, m_tiles - p.m_tile));
        linear_stream<T, MT, NT, ROWS><<<grid, kStreamThreads, sums > codes ? sums : codes, st>>>(p);
        e = hipGetLastError();
    }
    return e;
}
template <typename T, int MT, int ROWS> hipError_t launch_stream3(const StreamParams &p, hipStream_t st) {
    // 32 rows of w to a workgroup where that leaves two for every CU, else 16
    const bool two = (int64_t)((p.N + 31) / 32) * ((p.M + 16 * MT - 1) / (16 * MT)) >= 2 * kCus;
    return two ? launch_stream4<T, MT, 2, ROWS>(p, st) : launch_stream4<T, MT, 1, ROWS>(p, st);
}
template <typename T> hipError_t launch_stream(const LinearArgs &a, const CodesLayout &l, hipStream_t st) {
    const StreamParams p{l, a.w, a.w_scale, a.bias, a.x, a.x_stride, a.y, a.M, a.N, a.K, a.dtype, a.act, 0};
    if (!a.rows) switch (fused_rows(a.M, a.K)) {
        case 1: return launch_stream3<T, 1, 1>(p, st);
        case 2: return launch_stream3<T, 1, 2>(p, st);
        case 4: return launch_stream3<T, 1, 4>(p, st);
        case 8: return launch_stream3<T, 1, 8>(p, st);
        case 16: return launch_stream3<T, 1, 16>(p, st);
    }
    const hipError_t e = a.rows ? hipSuccess : launch_quant_rows(a, l, nullptr, nullptr, 0, st);
    if (e != hipSuccess) return e;
    // from here on x is not read: one type of the kernel serves all
    if (a.M <= 16) return launch_stream3<float, 1, 0>(p, st);
    if (a.M <= 32) return launch_stream3<float, 2, 0>(p, st);
    if (a.M <= 48) return launch_stream3<float, 3, 0>(p, st);
    return launch_stream3<float, 4, 0>(p, st);
}

template <typename T, bool SILU> hipError_t launch2(const LinearArgs &a, const CodesLayout &l, hipStream_t st) {
    const Kind kind = kind_of(a.M, a.N, a.K);
    const bool copy = needs_copy(a.M, a.N, a.K);
    // where only w's start is off 16 bytes there is no room for a copy
    if (kind == kStream || (!copy && (uintptr_t)a.w % 16 != 0)) return launch_stream<T>(a, l, st);
    TileParams p{l, a.w, a.K, a.w_scale, a.bias, a.y, a.M, a.N, 0, 0, 1, 0, nullptr, nullptr};
    const int steps = l.Kp / 128, splits = splits_of(a.M, a.N, a.K), count = (int)tiles(a.M, a.N, 64);
    p.split_steps = (steps + splits - 1) / splits;
    p.splits = (steps + p.split_steps - 1) / p.split_steps;
    int8_t *const beside = a.rows ? (int8_t *)a.workspace : l.codes + (int64_t)l.rows * l.Kp, *const to = copy ? beside : nullptr;
    p.sums = (int *)(beside + (copy ? (int64_t)a.N * l.Kp : 0));
    p.arrived = p.sums + (int64_t)splits * count * 4096;
    int *const zeros = p.splits > 1 ? p.arrived : nullptr;
    hipError_t e = hipSuccess;
    if (!a.rows) e = launch_quant_rows(a, l, to, zeros, count, st);
    else if (to || zeros) e = launch_beside_rows(a, l, to, zeros, count, st);
    if (e != hipSuccess) return e;
    if (copy) p.w = to, p.w_stride = l.Kp;
    const int b = kind == kTile256 ? 256 : kind == kRing128 ? 128 : 64;
    p.m_tiles = (a.M + b - 1) / b, p.n_tiles = (a.N + b - 1) / b;
    const dim3 grid(p.m_tiles * p.n_tiles, p.splits);
    if (kind == kTile256) linear_tile<T, SILU, 256, 256, 4><<<grid, 512, 0, st>>>(p);
    else if (kind == kRing128) linear_ring<T, SILU, 128, 128, 2><<<grid, 256, 0, st>>>(p);
    else linear_ring<T, SILU, 64, 64, 1><<<grid, 128, 0, st>>>(p);
    return hipGetLastError();
}
template <typename T> hipError_t launch1(const LinearArgs &a, const CodesLayout &l, hipStream_t st) {
    return a.act == CBS_ACT_SILU ? launch2<T, true>(a, l, st) : launch2<T, false>(a, l, st);
}

}  // namespace

int64_t linear_workspace(int64_t M, int64_t N, int64_t K, bool rows) {
    const CodesLayout l = codes_layout(nullptr, M, K);
    const int64_t splits = splits_of(M, N, K);
    return (rows ? 0 : l.bytes) + (needs_copy(M, N, K) ? N * l.Kp : 0) + (splits > 1 ? tiles(M, N, 64) * (splits * 16384 + 4) : 0);
}

hipError_t launch_int8_linear(const LinearArgs &a, hipStream_t st) {
    const CodesLayout l = codes_layout(a.rows ? const_cast<void *>(a.rows) : a.workspace, a.M, a.K);
    switch (a.dtype) {
        case CBS_DTYPE_F32: return launch1<float>(a, l, st);
        case CBS_DTYPE_BF16: return launch1<__bf16>(a, l, st);
        default: return launch1<_Float16>(a, l, st);
    }
}

}  // namespace cbs
