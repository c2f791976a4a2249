// k_attention_many.hip -- paged attention where a sequence has many rows: prompts
// and their chunks.  The work is the matrix products and the softmax between
// them.
//
// A workgroup takes a tile of rows, 32 to a wave, and goes through the keys 64 at
// a time.  Keys and values come through registers (where 8-bit codes become fp16,
// once for all the workgroup's rows) into two LDS buffers, so that one barrier a
// step suffices: while a step is computed, the loads of the next are on
// their way, and the page numbers of the one after.  A wave's scores never
// leave its registers.
//
// Bound by the issue of vector and matrix instructions, which hardly overlap (60% and 37% of
// a SIMD's cycles), and by power: 2 prompts of 8192, 32 heads over 8, dim 128, 8 bits: 1280
// us, 0.86 PFLOP/s; a large library product reaches 1.2.  Value scales that differ by more than 2^7
// within 64 keys, all along: 1725.
#include <hip/hip_runtime.h>

#include "b8_attention.h"

namespace cbs {
namespace {

constexpr int KT = 64;  // keys of a wave's step

// NB: dims in 32s.  SPLIT 2: half of the waves have the same rows as the other half and
// take every second 64 keys; the two meet at the end.  A tile has half of the rows then,
// and half of the steps in a row, for more bytes through LDS a row (a prompt of 1000, 32 heads
// over 8, 49.4 -> 36.0 us; of 4000, which fills the CUs without it, 167 and 211).
template <typename C, int NB, int SPLIT> struct ManyShape {
    static constexpr bool kI8 = std::is_same_v<C, int8_t>;
    // Dim 256 needs the registers of two waves; 16-bit caches at dim 64 need so few that three
    // waves fit a SIMD (2 prompts of 6000: 8 waves 469 us, 12 waves 407; with 8-bit
    // caches 543 and 593, for there it takes scratch memory or 168 registers of 192).
    static constexpr int kWaves = NB > 4 ? 4 : NB == 2 && !kI8 && SPLIT == 1 ? 12 : 8;
    // A wave at its step goes before one that stages the next (2 prompts of 8192, 8 bits, 1317 ->
    // 1302 us; 2 of 6000, 16 bits, 699 -> 689, dim 64 412 -> 401; 8 bits at dim 64 533 -> 551, dim
    // 256 2085 -> 2098).
    static constexpr bool kStepFirst = NB <= 4 && (NB > 2 || !kI8);
    static constexpr int kGroups = kWaves / SPLIT;  // waves with rows of their own
    static constexpr int kThreads = 64 * kWaves, kTile = 32 * kGroups, KS = KT * SPLIT;
    static constexpr int kPitchDims = NB <= 2 ? 64 : NB <= 4 ? 128 : 256;
    static constexpr int kPitch = 2 * kPitchDims;                         // bytes of a row in LDS
    static constexpr int kPieces = kPitchDims * (int)sizeof(C) / 16;      // 16-byte pieces of a row of the cache
    static constexpr int kRowsPerLoad = kThreads / kPieces;
    static constexpr int kLoads = kRowsPerLoad < KS ? KS / kRowsPerLoad : 1;
    static constexpr bool kIdle = kRowsPerLoad > KS;                      // threads without a piece
    static constexpr int kSide = KS * kPitch;                             // bytes of keys, or of values
    static constexpr int kOutPitch = kPitch + 16;
    static constexpr int kOutBytes = kTile * kOutPitch;
    static constexpr int kMeet = NB * 4096 + 512;  // bytes of a wave's outputs, maxima and sums
    static constexpr int kBytes = 4 * kSide > kOutBytes ? 4 * kSide : kOutBytes;
    static_assert(SPLIT == 1 || kGroups * kMeet <= kBytes, "");
    // Pieces of a row are exchanged: a read of keys takes the same dims of 16 rows at a
    // time, a transposed read of values 32 dims of 4 rows.
    static __device__ __forceinline__ int swap_k(int row) { return NB <= 2 ? (row >> 1) & 7 : row & 15; }
    static __device__ __forceinline__ int swap_v(int row) { return NB <= 2 ? (row & 2) << 1 : (row & 3) << 2; }
};

// Tile number `slot` of those that attend_many has, over all sequences.
struct Found {
    Sequence s;
    int tile;
};
__device__ __forceinline__ bool find_tile(const AttentionPlan &p, int slot, Found &f) {
    const int lane = (int)threadIdx.x % 64;
    int before = 0;
    for (int b0 = 0; b0 < p.a.batch; b0 += 64) {
        int tiles = 0;
        if (b0 + lane < p.a.batch) {
            const int rows = sequence(p, b0 + lane).n * (int)p.group.d;
            if (is_many(p, rows)) tiles = (rows + p.many.tile - 1) / p.many.tile;
        }
        int upto = tiles;
#pragma unroll
        for (int o = 1; o < 64; o *= 2) {
            const int x = __shfl_up(upto, o, 64);
            if (lane >= o) upto += x;
        }
        const uint64_t past = __ballot(before + upto > slot);
        if (past) {
            const int at = __builtin_ctzll(past);
            f.tile = slot - before - (__shfl(upto, at, 64) - __shfl(tiles, at, 64));
            f.tile = __builtin_amdgcn_readfirstlane(f.tile);
            f.s = sequence(p, __builtin_amdgcn_readfirstlane(b0 + at));
            return true;
        }
        before += __shfl(upto, 63, 64);
    }
    return false;
}

// The larger of a lane's value and that of the lane 32 away.
__device__ __forceinline__ float max_halves(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// Zeroes the infinities and NaN among 8 halves; whether there were any.
template <typename X> __device__ __forceinline__ bool take_out(u32x4 &v) {
    constexpr uint32_t kExp = std::is_same_v<X, _Float16> ? 0x7C00u : 0x7F80u;
    bool any = false;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const bool lo = (v[e] & kExp) == kExp, hi = ((v[e] >> 16) & kExp) == kExp;
        v[e] &= (lo ? 0u : 0xFFFFu) | (hi ? 0u : 0xFFFF0000u);
        any |= lo || hi;
    }
    return any;
}

template <typename T, typename C, int NB, int SPLIT>
__global__ __launch_bounds__((ManyShape<C, NB, SPLIT>::kThreads), (ManyShape<C, NB, SPLIT>::kWaves / 4)) void attend_many(const AttentionPlan p) {
    using S = ManyShape<C, NB, SPLIT>;
    constexpr int KS = S::KS;
    using X8 = typename Operand<T, C>::x8;
    using X = typename Operand<T, C>::type;
    constexpr int kSteps = 2 * NB, kAhead = 4;
    __shared__ __attribute__((aligned(16))) unsigned char lds[S::kBytes];
    __shared__ __attribute__((aligned(16))) float kscale[2][KS], vscale[2][KS];
    __shared__ uint64_t valid_bits[2][SPLIT];
    __shared__ float units[2][SPLIT];  // ValueUnit::of_tile
    __shared__ int taken_out[2][SPLIT];  // the last step in whose values store() found something to take out
    const AttentionArgs &a = p.a;
    const int tid = (int)threadIdx.x, lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64);
    const int part = SPLIT == 1 ? 0 : wave / S::kGroups, group = wave - part * S::kGroups;  // its keys of a step, its rows
    const int col = lane % 32, half = lane / 32;
    const int hk = a.cache.heads, dim = a.cache.dim;
    // the key/value head is innermost: with 8 of them each XCD's L2 serves one
    const int id = (int)blockIdx.x, kvh = id % hk, c = id / hk % p.many.chunks;
    Found f;
    // the last tiles of a sequence see the most keys: they go first
    if (!find_tile(p, p.slots - 1 - id / hk / p.many.chunks, f)) return;
    const Sequence &seq = f.s;
    const int rows = seq.n * (int)p.group.d;
    const int r0 = f.tile * S::kTile, r1 = min(rows, r0 + S::kTile);
    const Span2 keys = keys_of(p, seq, r0, r1);
    const int n_chunks = chunks_of(p.many, keys);
    if (c >= n_chunks) return;
    const int lo = keys.lo + c * p.many.chunk, hi = min(keys.hi, lo + p.many.chunk);
    const int old = seq.len - seq.n;
    // this wave's rows
    const int w0 = min(r0 + 32 * group, r1 - 1), w1 = min(r0 + 32 * group + 31, r1 - 1);
    const int wave_min = old + (int)p.group.div((uint32_t)w0), wave_max = old + (int)p.group.div((uint32_t)w1);
    const int wave_low = first_key(p, wave_min), wave_high_low = first_key(p, wave_max);

    const int32_t *const table = a.table + (int64_t)seq.b * a.table_stride;
    const C *const kdata = (const C *)a.cache.k, *const vdata = (const C *)a.cache.v;

    // this lane's row
    const int r = min(r0 + 32 * group + col, r1 - 1), tok = (int)p.group.div((uint32_t)r);
    const int pos = old + tok, low = first_key(p, pos);
    float qf = fmaxf(fabsf(a.scale) * kLog2e, 0x1p-149f);  // above zero, so that -inf stays what it is
    X8 q[kSteps];
    {
        const T *src = (const T *)a.q + (int64_t)(seq.first + tok) * a.q_token +
                       (int64_t)(kvh * (int)p.group.d + r - tok * (int)p.group.d) * a.q_head;
        const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;
        u32x4 raw[kSteps];
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int d = 16 * s + 8 * half;
            raw[s] = u32x4{0u, 0u, 0u, 0u};
            if (d < dim) raw[s] = ((const Any16 *)(src + d))->v ^ flip;
        }
        if constexpr (std::is_same_v<X, T>) {
#pragma unroll
            for (int s = 0; s < kSteps; ++s) q[s] = __builtin_bit_cast(X8, raw[s]);
        } else {
            uint32_t top = 0;
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
#pragma unroll
                for (int e = 0; e < 4; ++e) top = max(top, max(raw[s][e] & 0x7FFFu, (raw[s][e] >> 16) & 0x7FFFu));
            top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
            const int e = top >= 0x7F80u ? 0 : min(126, 141 - (int)(top >> 7));
            qf = fmaxf(__builtin_ldexpf(qf, -e), 0x1p-149f);
            const float up = __builtin_ldexpf(1.f, e);
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                const bf16x8 v = __builtin_bit_cast(bf16x8, raw[s]);
#pragma unroll
                for (int e8 = 0; e8 < 8; ++e8) q[s][e8] = (X)((float)v[e8] * up);
            }
        }
    }

    // Staging: thread's piece of rows my_row, my_row + kRowsPerLoad, ...; the first wave
    // also looks after the keys as such, one a lane: whether they are there, their scales.
    const bool my_part = !S::kIdle || tid / S::kPieces < KS;
    const int my_row = tid / S::kPieces % KS, my_d = tid % S::kPieces * (16 / (int)sizeof(C));
    const bool my_dims = my_d < dim;
    u32x4 kreg[S::kLoads], vreg[S::kLoads];
    bool vok[S::kLoads];
    int next_page[S::kLoads], key_page = -1;
    float ks = 0.f, vs = 0.f;
    ValueUnit value_unit;
    uint64_t key_bits = 0;
    auto page_of = [&](int j) { return j < hi ? table[p.page.div((uint32_t)j)] : -1; };
    auto row_of = [&](int j, int page, bool &ok) {
        ok = page >= 0 && page < a.cache.pages;
        const int off = j - (int)(p.page.div((uint32_t)j) * p.page.d);
        return ok ? ((int64_t)page * hk + kvh) * (int64_t)p.page.d + off : (int64_t)0;
    };
    auto look_up = [&](int j0) {
#pragma unroll
        for (int i = 0; i < S::kLoads; ++i) next_page[i] = page_of(j0 + my_row + i * S::kRowsPerLoad);
        if (group == 0) key_page = page_of(j0 + KT * part + lane);
    };
    auto load = [&](int j0) {
#pragma unroll
        for (int i = 0; i < S::kLoads; ++i) {
            const int64_t at = row_of(j0 + my_row + i * S::kRowsPerLoad, next_page[i], vok[i]) * dim + (my_dims ? my_d : 0);
            kreg[i] = *(const u32x4 *)(kdata + at);
            vreg[i] = *(const u32x4 *)(vdata + at);
        }
        if (group == 0) {
            bool ok;
            const int64_t row = row_of(j0 + KT * part + lane, key_page, ok);
            key_bits = __ballot(ok);
            if constexpr (S::kI8) {
                ks = a.cache.k_scale[row];
                vs = a.cache.v_scale[row];
            }
        }
    };
    // Values that only some of the tile's rows see may be infinite or NaN, and zero times
    // those is no zero: where some rows see a step in part, they are taken out here and
    // added apart.  8-bit codes are finite; their scales are taken out wherever they are not.
    const int tile_min = old + (int)p.group.div((uint32_t)r0);
    const int tile_low = first_key(p, old + (int)p.group.div((uint32_t)(r1 - 1)));
    auto store = [&](int buf, int j0) {
        unsigned char *const kbuf = lds + buf * 2 * S::kSide, *const vbuf = kbuf + S::kSide;
        const bool shared = j0 + KS - 1 > tile_min || j0 < tile_low;
        bool odd = false;
#pragma unroll
        for (int i = 0; i < S::kLoads; ++i) {
            const int row = my_row + i * S::kRowsPerLoad;
            const u32x4 k = kreg[i];
            if (!my_part) continue;
            if constexpr (S::kI8) {
                const u32x4 v = vreg[i];
                // 16 codes: two pieces of a row in LDS
                const int piece = 2 * (tid % S::kPieces);
                unsigned char *const kr = kbuf + row * S::kPitch, *const vr = vbuf + row * S::kPitch;
                *(f16x8 *)(kr + ((piece ^ S::swap_k(row)) * 16)) = codes_f16(k[0], k[1]);
                *(f16x8 *)(kr + (((piece + 1) ^ S::swap_k(row)) * 16)) = codes_f16(k[2], k[3]);
                *(f16x8 *)(vr + ((piece ^ S::swap_v(row)) * 16)) = codes_f16(v[0], v[1]);
                *(f16x8 *)(vr + (((piece + 1) ^ S::swap_v(row)) * 16)) = codes_f16(v[2], v[3]);
            } else {
                const int piece = tid % S::kPieces;
                // past dim q is zero, and a key's infinity or NaN has no place there
                const uint32_t kkeep = my_dims ? ~0u : 0u, vkeep = vok[i] ? ~0u : 0u;
                u32x4 v = vreg[i] & vkeep;
                if (shared) odd |= take_out<X>(v);
                *(u32x4 *)(kbuf + row * S::kPitch + ((piece ^ S::swap_k(row)) * 16)) = k & kkeep;
                *(u32x4 *)(vbuf + row * S::kPitch + ((piece ^ S::swap_v(row)) * 16)) = v;
            }
        }
        if constexpr (!S::kI8) {
            if (__any(odd) && lane < SPLIT) taken_out[buf][lane] = j0;
        }
        if (group == 0) {
            if constexpr (S::kI8) {
                const uint32_t bits = magnitude(vs);
                const bool there = (key_bits >> lane) & 1, counts = there && bits < 0x7F800000u;
                const uint64_t taken = __ballot(there && !counts);
                if (taken && lane == 0) taken_out[buf][part] = j0;
                if (!counts) vs = 0.f;
                const float unit = value_unit.of_tile(bits, counts);
                kscale[buf][KT * part + lane] = finite_or_nan(ks);
                vscale[buf][KT * part + lane] = in_unit(vs, unit);
                if (lane == 0) units[buf][part] = unit;
            }
            if (lane == 0) valid_bits[buf][part] = key_bits;
        }
    };

    // where the lane's reads of a buffer's keys and values begin
    const int k_lane = col * S::kPitch + ((half ^ S::swap_k(col)) * 16), v_row = 4 * half + lane % 16 / 4;
    const int v_lane = v_row * S::kPitch + (((2 * (lane / 16 % 2) + lane % 4 / 2) ^ S::swap_v(v_row)) * 16) + lane % 2 * 8;

    f32x16 o[NB] = {};
    // 8-bit caches: m and mo are exponents; else m is a score, and the outputs are in its unit
    float m = S::kI8 ? kNoExponent : -INFINITY, l = 0.f, mo = kNoExponent;

    if (tid < 2 * SPLIT) taken_out[tid / SPLIT][tid % SPLIT] = -1;
    __syncthreads();
    if (lo < hi) {
        look_up(lo);
        load(lo);
        look_up(lo + KS);
        store(0, lo);
    }
    int buf = 0;
    for (int j0 = lo; j0 < hi; j0 += KS, buf ^= 1) {
        __syncthreads();
        const bool more = j0 + KS < hi;
        const int jw = j0 + KT * part;
        if (more) {
            load(j0 + KS);
            if (j0 + 2 * KS < hi) look_up(j0 + 2 * KS);
        }
        if (jw < hi && jw <= wave_max && jw + KT > wave_low) {
            // An operand's piece number is exchanged by exclusive or, and so is its byte: one
            // operation for a step of the scores or a block of the outputs, and the rest is
            // the instruction's offset.
            int k_at = buf * 2 * S::kSide + part * KT * S::kPitch + k_lane, v_at = k_at - k_lane + S::kSide + v_lane;
            asm volatile("" : "+v"(k_at), "+v"(v_at));  // made anew for each step, or each costs a register
            // Fragments are read kAhead matrix instructions before their use, and the order is
            // held: left alone the compiler reads each just before it is wanted, and waits.
            auto read_k = [&](int i) { return *(const X8 *)(lds + (k_at ^ (32 * (i / 2))) + 32 * (i % 2) * S::kPitch); };
            f32x16 s[2];
            if (S::kStepFirst) __builtin_amdgcn_s_setprio(1);
            X8 ring[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) ring[i] = read_k(i);
#pragma unroll
            for (int i = 0; i < 2 * kSteps; ++i) {
                __builtin_amdgcn_sched_barrier(0);
                s[i % 2] = mma32(ring[i % kAhead], q[i / 2], i < 2 ? f32x16{} : s[i % 2]);
                if (i + kAhead < 2 * kSteps) ring[i % kAhead] = read_k(i + kAhead);
            }
            const uint64_t valid = valid_bits[buf][part];
            // the lane's keys are 32 kb + 8 g + 4 half + 0..3
            f32x4 per_key[8];
            if constexpr (S::kI8) {
#pragma unroll
                for (int g = 0; g < 8; ++g) per_key[g] = *(const f32x4 *)(&kscale[buf][KT * part + 8 * g + 4 * half]);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int i = 0; i < 32; ++i) s[i / 16][i % 16] *= per_key[i / 4][i % 4];
            }
            if (!(valid == ~0ull && jw + KT - 1 <= wave_min && jw >= wave_high_low)) {
                int my_half = half;
                asm volatile("" : "+v"(my_half));
                const uint64_t ahead = valid >> (4 * my_half);
                const int last = pos - jw - 4 * my_half, first = low - jw - 4 * my_half;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const int key = 32 * (i / 16) + 8 * (i % 16 / 4) + i % 4;  // less 4 half
                    if (!(((ahead >> key) & 1) && key <= last && key >= first)) s[i / 16][i % 16] = -INFINITY;
                }
            }
            float tops[2] = {s[0][0], s[1][0]};
#pragma unroll
            for (int i = 1; i < 15; i += 2)
#pragma unroll
                for (int kb = 0; kb < 2; ++kb) tops[kb] = fmaxf(fmaxf(tops[kb], s[kb][i]), s[kb][i + 1]);
            const float top = max_halves(fmaxf(fmaxf(fmaxf(tops[0], s[0][15]), tops[1]), s[1][15]));
            float base, to_sum = 1.f;
            if constexpr (S::kI8) {
                const float unit = units[buf][part], x = top * qf;
#pragma unroll
                for (int g = 0; g < 8; ++g) per_key[g] = *(const f32x4 *)(&vscale[buf][KT * part + 8 * g + 4 * half]);
                const bool uneven = __builtin_amdgcn_readfirstlane(__float_as_int(unit)) == __builtin_bit_cast(int, kUneven);
                float u = x + unit;
                if (__builtin_expect(uneven, 0)) {
                    u = -INFINITY;
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        u = fmaxf(u, __builtin_fmaf(s[i / 16][i % 16], qf, __builtin_amdgcn_logf(fabsf(per_key[i / 4][i % 4]))));
                    u = max_halves(u);
                }
                if (__any(x > m + kSlack || u > mo + (kSlack + kLift))) {
                    const float now = x > m + kSlack ? x : m, now_o = product_exponent(mo, u);
                    l *= __builtin_amdgcn_exp2f(m - now);
                    const float fade = __builtin_amdgcn_exp2f(mo - now_o);
                    m = now, mo = now_o;
#pragma unroll
                    for (int db = 0; db < NB; ++db) o[db] *= fade;
                }
                base = tile_exponent(m, mo, unit);
                if (__builtin_expect(uneven, 0)) {
                    base = m;
#pragma unroll
                    for (int i = 0; i < 32; ++i) per_key[i / 4][i % 4] = uneven_scale(per_key[i / 4][i % 4], m, mo);
                }
                to_sum = __builtin_amdgcn_exp2f(base - m);
            } else {
                const bool move = top > m && !((top - m) * qf <= kSlack);
                if (__any(move)) {
                    const float now = move ? top : m;
                    const float fade = move ? (m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((m - now) * qf)) : 1.f;
                    m = now;
                    l *= fade;
#pragma unroll
                    for (int db = 0; db < NB; ++db) o[db] *= fade;
                }
                base = m == -INFINITY ? 0.f : __builtin_fmaf(m, qf, -kLiftOf<X>);
            }
            // values: keys 16 t + 4 half + 0..3 and 8 above those, of dim 32 db + col
            auto read_v = [&](int i) {
                const unsigned char *from = lds + (v_at ^ (64 * (i % NB))) + 16 * (i / NB) * S::kPitch;
                const u32x2 x = read_tr16(from), y = read_tr16(from + 8 * S::kPitch);
                return __builtin_bit_cast(X8, u32x4{x.x, x.y, y.x, y.y});
            };
#pragma unroll
            for (int i = 0; i < kAhead; ++i) ring[i] = read_v(i);
            __builtin_amdgcn_sched_barrier(0);
            // a key that is not seen: 2^-inf = 0
            float sums[2] = {0.f, 0.f};
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                X8 pr;
#pragma unroll
                for (int i = 8 * t; i < 8 * t + 8; ++i) {
                    float w = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i / 16][i % 16], qf, -base));
                    sums[i % 2] += w;
                    if constexpr (S::kI8) w *= per_key[i / 4][i % 4];
                    pr[i % 8] = (X)w;
                }
                // these keys' matrix instructions run beside the next ones' exponentials
#pragma unroll
                for (int i = NB * t; i < NB * t + NB; ++i) {
                    __builtin_amdgcn_sched_barrier(0);
                    o[i % NB] = mma32(ring[i % kAhead], pr, o[i % NB]);
                    if (i + kAhead < 4 * NB) ring[i % kAhead] = read_v(i + kAhead);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            if (S::kStepFirst) __builtin_amdgcn_s_setprio(0);
            l += (sums[0] + sums[1]) * to_sum;
            if (__builtin_expect(taken_out[buf][part] == j0, 0)) {
                // what store() has taken out, to the rows that see it
#pragma unroll 1
                for (int j = jw; j < min(hi, jw + KT); ++j) {
                    bool there;
                    const int64_t row = row_of(j, table[p.page.div((uint32_t)j)], there);
                    const bool sees = there && j <= pos && j >= low;
                    if constexpr (S::kI8) {
                        if (__builtin_isfinite(a.cache.v_scale[row])) continue;
                    }
#pragma unroll
                    for (int db = 0; db < NB; ++db)
#pragma unroll
                        for (int g = 0; g < 4; ++g) {
                            const int d = 32 * db + 8 * g + 4 * half;
                            if (d >= dim || !sees) continue;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                float v = (float)vdata[row * dim + d + e];
                                if constexpr (S::kI8) v *= a.cache.v_scale[row];
                                if (!__builtin_isfinite(v)) o[db][4 * g + e] += v;
                            }
                        }
                }
            }
        }
        if (more) store(buf ^ 1, j0 + KS);
    }

    // the lane has one row, of every 32 dims 16
    float ref = 1.f, top;  // the outputs' unit in that of the sum, whose exponent is top
    if constexpr (S::kI8) ref = __builtin_amdgcn_exp2f(mo - m), top = m == kNoExponent ? -INFINITY : m;
    else top = m == -INFINITY ? -INFINITY : m * qf;
    if constexpr (SPLIT == 2) {
        // the second half of the waves hand theirs over, lane by lane
        __syncthreads();
        float *const meet = (float *)(lds + group * S::kMeet), *const meet_ml = meet + NB * 1024;
        if (part == 1) {
#pragma unroll
            for (int x = 0; x < 4 * NB; ++x) {
                const f32x4 v = {o[x / 4][x % 4 * 4], o[x / 4][x % 4 * 4 + 1], o[x / 4][x % 4 * 4 + 2], o[x / 4][x % 4 * 4 + 3]};
                *(f32x4 *)(meet + (x * 64 + lane) * 4) = v * ref;
            }
            meet_ml[lane] = top, meet_ml[64 + lane] = l;
        }
        __syncthreads();
        if (part == 0) {
            const float other = meet_ml[lane], both_top = fmaxf(top, other);
            const float mine = top == both_top ? 1.f : __builtin_amdgcn_exp2f(top - both_top);
            const float theirs = other == both_top ? 1.f : __builtin_amdgcn_exp2f(other - both_top);
            l = l * mine + meet_ml[64 + lane] * theirs;
            const float scale = mine * ref;
#pragma unroll
            for (int x = 0; x < 4 * NB; ++x) {
                const f32x4 v = *(const f32x4 *)(meet + (x * 64 + lane) * 4);
#pragma unroll
                for (int e = 0; e < 4; ++e) o[x / 4][x % 4 * 4 + e] = o[x / 4][x % 4 * 4 + e] * scale + v[e] * theirs;
            }
            ref = 1.f, top = both_top;
        }
    }
    const auto both = __builtin_amdgcn_permlane32_swap(__float_as_uint(l), __float_as_uint(l), false, false);
    const float sum = __uint_as_float(both[0]) + __uint_as_float(both[1]);
    // Through LDS, so that a row's dims are stored side by side; parts, in fp32, half of them at a time.
    __syncthreads();
    if (part != 0) return;
    unsigned char *const stage = lds + group * 32 * S::kOutPitch;
    constexpr int kOutPieces = S::kPitch / 16;
    if (n_chunks > 1) {
        constexpr int kHalf = S::kPitchDims / 2;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int db = 0; db < NB; ++db)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    if (32 * db / kHalf != h) continue;
                    const f32x4 v = {o[db][4 * g], o[db][4 * g + 1], o[db][4 * g + 2], o[db][4 * g + 3]};
                    *(f32x4 *)(stage + col * S::kOutPitch + 4 * (32 * db - h * kHalf + 8 * g + 4 * half)) = v * ref;
                }
            __builtin_amdgcn_wave_barrier();
#pragma unroll 1
            for (int i = lane; i < 32 * kOutPieces; i += 64) {
                const int row = i / kOutPieces, d = h * kHalf + i % kOutPieces * 4, at = r0 + 32 * group + row;
                if (at < r1 && d < dim)
                    *(f32x4 *)(p.many.o + (out_line(p, seq, kvh, at) * p.many.room + c) * dim + d) =
                        *(const f32x4 *)(stage + row * S::kOutPitch + i % kOutPieces * 16);
            }
            __builtin_amdgcn_wave_barrier();
        }
        const int mine = r0 + 32 * group + col;
        if (half == 0 && mine < r1) {
            const int64_t line = out_line(p, seq, kvh, mine) * p.many.room + c;
            p.many.ml[2 * line] = top, p.many.ml[2 * line + 1] = sum;
        }
        return;
    }
#pragma unroll
    for (int db = 0; db < NB; ++db)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            typedef T x4 __attribute__((ext_vector_type(4)));
            x4 v;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = (T)(divide(o[db][4 * g + e], sum) * ref);
            *(x4 *)(stage + col * S::kOutPitch + 2 * (32 * db + 8 * g + 4 * half)) = v;
        }
    __builtin_amdgcn_wave_barrier();
#pragma unroll 1
    for (int i = lane; i < 32 * kOutPieces; i += 64) {
        const int row = i / kOutPieces, d = i % kOutPieces * 8, at = r0 + 32 * group + row;
        if (at < r1 && d < dim)
            ((Any16 *)((T *)a.out + out_line(p, seq, kvh, at) * dim + d))->v = *(const u32x4 *)(stage + row * S::kOutPitch + 2 * d);
    }
}

template <typename T, typename C, int NB, int SPLIT> hipError_t launch4(const AttentionPlan &p, hipStream_t st) {
    const int64_t grid = (int64_t)p.slots * p.many.chunks * p.a.cache.heads;
    attend_many<T, C, NB, SPLIT><<<(unsigned)grid, ManyShape<C, NB, SPLIT>::kThreads, 0, st>>>(p);
    return hipGetLastError();
}
template <typename T, typename C, int NB> hipError_t launch3(const AttentionPlan &p, hipStream_t st) {
    return p.split ? launch4<T, C, NB, 2>(p, st) : launch4<T, C, NB, 1>(p, st);
}
template <typename T, typename C> hipError_t launch2(const AttentionPlan &p, hipStream_t st) {
    if (p.a.cache.dim <= 64) return launch3<T, C, 2>(p, st);
    if (p.a.cache.dim <= 96) return launch3<T, C, 3>(p, st);
    return p.a.cache.dim <= 128 ? launch3<T, C, 4>(p, st) : launch4<T, C, 8, 1>(p, st);
}
template <typename T> hipError_t launch1(const AttentionPlan &p, hipStream_t st) {
    return p.a.cache.dtype == CBS_DTYPE_I8 ? launch2<T, int8_t>(p, st) : launch2<T, T>(p, st);
}

}  // namespace

int many_tile(int64_t dim, bool int8, bool split) {
    if (dim > 128) return ManyShape<int8_t, 8, 1>::kTile;
    if (split) return ManyShape<int8_t, 4, 2>::kTile;
    return dim <= 64 && !int8 ? ManyShape<__bf16, 2, 1>::kTile : ManyShape<int8_t, 4, 1>::kTile;
}

hipError_t launch_attend_many(const AttentionPlan &p, hipStream_t st) {
    return p.a.dtype == CBS_DTYPE_BF16 ? launch1<__bf16>(p, st) : launch1<_Float16>(p, st);
}

}  // namespace cbs
