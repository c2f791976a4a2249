// k_attention_few.hip -- paged attention where a sequence has few rows: single
// tokens above all.  The work is the reading of the cache, so it is divided
// along the keys: first into chunks, one to a workgroup, then into tiles of KT
// keys that the waves of a workgroup take in turn, each with its own running
// maximum, sum and output.  They meet in LDS at the end, and the chunks through
// the workspace.
//
// A wave streams: while it works on one tile the next one's keys, values and
// scales are on their way into registers (16 KiB a wave at dim 128, eight waves a
// CU: more than the CU needs outstanding to draw its share of HBM), and the page
// numbers of the one after that.  Keys go from registers into the matrix
// instructions as they are; values pass through a piece of LDS that only the wave uses, and
// come back transposed.  No barrier in the loop.
//
// Bound by HBM: 64 sequences of 2000 to 16000 keys, 32 heads over 8, dim 128, 8 bits: 244 us a
// call, 5.0 TB/s (16 bits: 428 us, 5.5 TB/s; a large copy reaches 6.3; dim 256: 521 and 839 us).  Value
// scales that differ by more than 2^7 within 64 keys cost 20 us of 244.  The matrix pipe is 7%
// busy, though 12 of its 16 columns are padding there, and the vector pipe 49%: what
// unpacks the codes and the softmax hides under the loads.
#include <hip/hip_runtime.h>

#include "b8_attention.h"

namespace cbs {
namespace {

constexpr int kWaves = 4, kThreads = 64 * kWaves;

template <typename C, int ND, int QT> struct FewShape {
    static constexpr bool kI8 = std::is_same_v<C, int8_t>;
    static constexpr int kDims = 64 * ND;                   // dims, padded
    static constexpr int KT = kI8 && ND <= 2 ? 64 : 32;     // keys of a tile
    static constexpr int kRow = kDims * (int)sizeof(C);     // bytes of a row of values in LDS
    static constexpr int kPieces = kRow / 16;               // 16-byte pieces of it
    static constexpr int kLoads = KT * kRow / 1024;         // a wave's 16-byte loads of a tile
    static constexpr int kRowsPerLoad = 64 / kPieces;
    static constexpr int kSteps = kDims / 32;               // matrix steps of the scores
    // two waves a SIMD where the registers allow (256 a wave), else one
    static constexpr int kPerSimd = ND <= 2 && QT * ND <= 2 ? 2 : 1;
    static constexpr int kWaveBytes = KT * kRow + KT * 8 + 2 * KT * 4;
    static constexpr int kOutPitch = kDims + 4;             // floats
    static constexpr int kOutBytes = kWaves * 16 * QT * (kOutPitch + 2) * 4;
    static constexpr int kBytes = kWaves * kWaveBytes > kOutBytes ? kWaves * kWaveBytes : kOutBytes;
    // Pieces of a row are exchanged so that a transposed read, which takes the same columns
    // of 8 rows (of 16 for 8-bit codes) at a time, finds them in different banks.
    static __device__ __forceinline__ int swap(int row) {
        if constexpr (kI8) {
            const int far = (row >> 4) & 1;
            if constexpr (ND == 1) return ((row >> 2) & 1) | far << 1;
            else if constexpr (ND == 2) return ((row >> 1) & 3) | far << 2;
            else return (row & 7) | far << 3;
        } else {
            return ND == 1 ? ((row >> 1) & 3) * 2 : (row & 7) * 2;
        }
    }
};

template <typename T, typename C, int ND, int QT>
__global__ __launch_bounds__(kThreads, (FewShape<C, ND, QT>::kPerSimd)) void attend_few(const AttentionPlan p) {
    using S = FewShape<C, ND, QT>;
    using X8 = typename Operand<T, C>::x8;
    using X = typename Operand<T, C>::type;
    constexpr int KT = S::KT, KB = KT / 16;
    constexpr uint64_t kAll = KT == 64 ? ~0ull : (1ull << (KT % 64)) - 1;
    __shared__ __attribute__((aligned(16))) unsigned char lds[S::kBytes];
    const AttentionArgs &a = p.a;
    const int lane = (int)threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / 64);
    const int col = lane % 16, grp = lane / 16;
    const int hk = a.cache.heads, dim = a.cache.dim;
    const int id = (int)blockIdx.x, kvh = id % hk, at = id / hk, b = at % a.batch, c = at / a.batch;
    const Sequence seq = sequence(p, b);
    const int rows = seq.n * (int)p.group.d;
    if (rows == 0 || is_many(p, rows)) return;

    unsigned char *const vbuf = lds + wave * S::kWaveBytes;
    int64_t *const place = (int64_t *)(vbuf + KT * S::kRow);   // of the tile's keys: their row of the cache
    float *const kscale = (float *)(place + KT), *const vscale = kscale + KT;
    const int32_t *const table = a.table + (int64_t)b * a.table_stride;
    const C *const kdata = (const C *)a.cache.k, *const vdata = (const C *)a.cache.v;
    const float c0 = fabsf(a.scale) * kLog2e;

    for (int r0 = 0; r0 < rows; r0 += 16 * QT) {
        const int r1 = min(rows, r0 + 16 * QT);
        const Span2 keys = keys_of(p, seq, r0, r1);
        const int n_chunks = chunks_of(p.few, keys);
        if (c >= n_chunks) continue;
        const int lo = keys.lo + c * p.few.chunk, hi = min(keys.hi, lo + p.few.chunk);
        const int pos_min = seq.len - seq.n + (int)p.group.div((uint32_t)r0);
        const int pos_max = seq.len - seq.n + (int)p.group.div((uint32_t)(r1 - 1));

        // this lane's rows: the positions they stand at, what they see, their queries
        int pos[QT], low[QT];
        float qf[QT];
        X8 q[QT][S::kSteps];
#pragma unroll
        for (int i = 0; i < QT; ++i) {
            const int r = min(r0 + 16 * i + col, r1 - 1), tok = (int)p.group.div((uint32_t)r);
            pos[i] = seq.len - seq.n + tok;
            low[i] = first_key(p, pos[i]);
            const T *src = (const T *)a.q + (int64_t)(seq.first + tok) * a.q_token +
                           (int64_t)(kvh * (int)p.group.d + r - tok * (int)p.group.d) * a.q_head;
            // the dims of step s that this group of lanes holds, as the keys' loads hand them out
            auto dims = [&](int s) { return S::kI8 ? (s / 2) * 64 + grp * 16 + (s % 2) * 8 : s * 32 + grp * 8; };
            const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;
            u32x4 raw[S::kSteps];
#pragma unroll
            for (int s = 0; s < S::kSteps; ++s) {
                raw[s] = u32x4{0u, 0u, 0u, 0u};
                if (dims(s) < dim) raw[s] = ((const Any16 *)(src + dims(s)))->v ^ flip;
            }
            qf[i] = fmaxf(c0, 0x1p-149f);  // above zero, so that -inf stays what it is
            if constexpr (std::is_same_v<X, T>) {
#pragma unroll
                for (int s = 0; s < S::kSteps; ++s) q[i][s] = __builtin_bit_cast(X8, raw[s]);
            } else {
                uint32_t top = 0;
#pragma unroll
                for (int s = 0; s < S::kSteps; ++s)
#pragma unroll
                    for (int e = 0; e < 4; ++e) top = max(top, max(raw[s][e] & 0x7FFFu, (raw[s][e] >> 16) & 0x7FFFu));
                top = max(top, (uint32_t)__shfl_xor((int)top, 16, 64));
                top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
                // exponent 14 for the largest; rows of infinities and NaN stay as they are
                const int e = top >= 0x7F80u ? 0 : min(126, 141 - (int)(top >> 7));
                qf[i] = fmaxf(__builtin_ldexpf(c0, -e), 0x1p-149f);
                const float up = __builtin_ldexpf(1.f, e);
#pragma unroll
                for (int s = 0; s < S::kSteps; ++s) {
                    const bf16x8 v = __builtin_bit_cast(bf16x8, raw[s]);
#pragma unroll
                    for (int e8 = 0; e8 < 8; ++e8) q[i][s][e8] = (X)((float)v[e8] * up);
                }
            }
        }

        f32x4 o[QT][S::kDims / 16] = {};
        // 8-bit caches: m and mo are exponents; else m is a score, and the outputs are in its unit
        float m[QT], l[QT], mo[QT];
#pragma unroll
        for (int i = 0; i < QT; ++i) m[i] = S::kI8 ? kNoExponent : -INFINITY, mo[i] = kNoExponent, l[i] = 0.f;
        ValueUnit units;

        // the tile in registers, and what belongs to it; lane i has key j0 + i
        u32x4 kreg[KB][S::kRow / 64], vreg[S::kLoads];
        float ks = 0.f, vs = 0.f;
        uint64_t there = 0;  // bit i: key i of the tile in registers is in the cache
        auto page_of = [&](int j0) {
            const int j = j0 + lane % KT;
            return j < hi ? table[p.page.div((uint32_t)j)] : -1;
        };
        auto locate = [&](int j0, int page) {
            const int j = j0 + lane % KT;
            const bool ok = page >= 0 && page < a.cache.pages;
            const int off = j - (int)(p.page.div((uint32_t)j) * p.page.d);
            const int64_t row = ok ? ((int64_t)page * hk + kvh) * (int64_t)p.page.d + off : 0;
            place[lane % KT] = row;
            there = __ballot(ok) & kAll;
            if constexpr (S::kI8) {
                ks = a.cache.k_scale[row];
                vs = a.cache.v_scale[row];
            }
            __builtin_amdgcn_wave_barrier();
        };
        auto load_k = [&] {
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                const C *from = kdata + place[16 * kb + col] * dim;
#pragma unroll
                for (int s = 0; s < S::kRow / 64; ++s) {
                    const int d = (s * 64 + grp * 16) / (int)sizeof(C);
                    kreg[kb][s] = *(const u32x4 *)(from + (d < dim ? d : 0));
                }
            }
        };
        auto load_v = [&] {
#pragma unroll
            for (int i = 0; i < S::kLoads; ++i) {
                const int row = i * S::kRowsPerLoad + lane / S::kPieces, d = lane % S::kPieces * (16 / (int)sizeof(C));
                const C *from = vdata + place[row] * dim;
                vreg[i] = *(const u32x4 *)(from + (d < dim ? d : 0));  // past dim: outputs that are not stored
            }
        };

        const int step = kWaves * KT;
        int j0 = lo + wave * KT;
        if (j0 < hi) {
            locate(j0, page_of(j0));
            load_k();
            load_v();
        }
        int next_page = j0 + step < hi ? page_of(j0 + step) : -1;
        for (; j0 < hi; j0 += step) {
            const uint64_t valid = there;
            // scores; past dim, where q is zero, a number of the row would do, but not infinity or NaN
            f32x4 s[QT][KB] = {};
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                for (int st = 0; st < S::kSteps; ++st) {
                    X8 kf;
                    if constexpr (S::kI8) kf = codes_f16(kreg[kb][st / 2][st % 2 * 2], kreg[kb][st / 2][st % 2 * 2 + 1]);
                    else kf = __builtin_bit_cast(X8, kreg[kb][st] & (st * 32 + grp * 8 < dim ? ~0u : 0u));
#pragma unroll
                    for (int i = 0; i < QT; ++i) s[i][kb] = mma16(kf, q[i][st], s[i][kb]);
                }
            // this tile's scales and values to LDS, the next tile's on their way
            float unit = 0.f;
            bool uneven = false;
            if constexpr (S::kI8) {
                const uint32_t bits = magnitude(vs);
                unit = units.of_tile(bits, ((valid >> (lane % KT)) & 1) && bits < 0x7F800000u);
                uneven = __builtin_amdgcn_readfirstlane(__float_as_int(unit)) == __builtin_bit_cast(int, kUneven);
                kscale[lane % KT] = finite_or_nan(ks);
                vscale[lane % KT] = in_unit(vs, unit);
            }
            // LDS addresses are made anew for each tile: kept, they cost a register for each access
            int my = lane, my_col = col;
            asm volatile("" : "+v"(my), "+v"(my_col));
#pragma unroll
            for (int i = 0; i < S::kLoads; ++i) {
                const int row = i * S::kRowsPerLoad + my / S::kPieces, piece = (my % S::kPieces) ^ S::swap(row);
                *(u32x4 *)(vbuf + row * S::kRow + piece * 16) = vreg[i];
            }
            const int j1 = j0 + step;
            if (j1 < hi) {
                locate(j1, next_page);
                load_k();
                load_v();
                if (j1 + step < hi) next_page = page_of(j1 + step);
            }
            __builtin_amdgcn_wave_barrier();

            // softmax
            const bool full = valid == kAll && j0 + KT - 1 <= pos_min && j0 >= first_key(p, pos_max);
            X8 pr[QT][KT / 32];
            f32x4 vsc[KB];
            uint32_t seen[QT][KB];  // 4 bits: the lane's keys of a block that the row sees
            if constexpr (S::kI8) {
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
                    const f32x4 k4 = *(const f32x4 *)(kscale + 16 * kb + 4 * grp);
                    vsc[kb] = *(const f32x4 *)(vscale + 16 * kb + 4 * grp);
#pragma unroll
                    for (int i = 0; i < QT; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[i][kb][e] *= k4[e];
                }
            }
#pragma unroll
            for (int i = 0; i < QT; ++i) {
                if (!full) {
                    const uint64_t ahead = valid >> (4 * grp);
                    const int last = pos[i] - j0 - 4 * grp, first = low[i] - j0 - 4 * grp;
#pragma unroll
                    for (int kb = 0; kb < KB; ++kb) {
                        seen[i][kb] = 0;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int key = 16 * kb + e;  // less 4 grp
                            const bool see = ((ahead >> key) & 1) && key <= last && key >= first;
                            seen[i][kb] |= see ? 1u << e : 0u;
                            if (!see) s[i][kb][e] = -INFINITY;
                        }
                    }
                }
                float top = fmaxf(fmaxf(s[i][0][0], s[i][0][1]), fmaxf(s[i][0][2], s[i][0][3]));
#pragma unroll
                for (int kb = 1; kb < KB; ++kb)
                    top = fmaxf(top, fmaxf(fmaxf(s[i][kb][0], s[i][kb][1]), fmaxf(s[i][kb][2], s[i][kb][3])));
                top = fmaxf(top, __shfl_xor(top, 16, 64));
                top = fmaxf(top, __shfl_xor(top, 32, 64));
                float base, to_sum = 1.f;
                if constexpr (S::kI8) {
                    const float x = top * qf[i];
                    float u = x + unit;
                    if (uneven) {
                        u = -INFINITY;
#pragma unroll
                        for (int kb = 0; kb < KB; ++kb) {
                            __builtin_amdgcn_sched_barrier(0);  // rare: no registers to work on several at once
                            const f32x4 v = *(const f32x4 *)(vscale + 16 * kb + 4 * grp);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                u = fmaxf(u, __builtin_fmaf(s[i][kb][e], qf[i], __builtin_amdgcn_logf(fabsf(v[e]))));
                        }
                        u = fmaxf(u, __shfl_xor(u, 16, 64));
                        u = fmaxf(u, __shfl_xor(u, 32, 64));
                    }
                    if (__any(x > m[i] + kSlack || u > mo[i] + (kSlack + kLift))) {
                        const float now = x > m[i] + kSlack ? x : m[i], now_o = product_exponent(mo[i], u);
                        l[i] *= __builtin_amdgcn_exp2f(m[i] - now);
                        const float fade = __builtin_amdgcn_exp2f(mo[i] - now_o);
                        m[i] = now, mo[i] = now_o;
#pragma unroll
                        for (int d = 0; d < S::kDims / 16; ++d) o[i][d] *= fade;
                    }
                    base = tile_exponent(m[i], mo[i], unit);
                    if (uneven) {
                        base = m[i];
#pragma unroll
                        for (int kb = 0; kb < KB; ++kb) {
                            __builtin_amdgcn_sched_barrier(0);
                            vsc[kb] = *(const f32x4 *)(vscale + 16 * kb + 4 * grp);
#pragma unroll
                            for (int e = 0; e < 4; ++e) vsc[kb][e] = uneven_scale(vsc[kb][e], m[i], mo[i]);
                        }
                    }
                    to_sum = __builtin_amdgcn_exp2f(base - m[i]);
                } else {
                    const bool move = top > m[i] && !((top - m[i]) * qf[i] <= kSlack);
                    if (__any(move)) {
                        const float now = move ? top : m[i];
                        const float fade = move ? (m[i] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((m[i] - now) * qf[i])) : 1.f;
                        m[i] = now;
                        l[i] *= fade;
#pragma unroll
                        for (int d = 0; d < S::kDims / 16; ++d) o[i][d] *= fade;
                    }
                    base = m[i] == -INFINITY ? 0.f : __builtin_fmaf(m[i], qf[i], -kLiftOf<X>);
                }
                float sum = 0.f;
#pragma unroll
                for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float w = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i][kb][e], qf[i], -base));
                        if (!full && !((seen[i][kb] >> e) & 1)) w = 0.f;
                        sum += w;
                        if constexpr (S::kI8) {
                            w *= vsc[kb][e];
                            if (!full && !((seen[i][kb] >> e) & 1)) w = 0.f;  // the scale may be anything
                        }
                        pr[i][kb / 2][kb % 2 * 4 + e] = (X)w;
                    }
                l[i] += sum * to_sum;
            }

            // values: keys 32 t + 4 grp + 0..3 and 16 above those, of dim 16 db + col
            auto values = [&](int db, int t) {
                u32x4 v;
                if constexpr (S::kI8) {
                    const int r = my_col / 2, row = 32 * t + 4 * grp + r % 4 + 16 * (r / 4);
                    const u32x2 x = read_tr8(vbuf + row * S::kRow + ((db ^ S::swap(row)) * 16) + my_col % 2 * 8);
                    v = __builtin_bit_cast(u32x4, codes_f16(x.x, x.y));
                } else {
                    const int row = 32 * t + 4 * grp + my_col / 4, piece = (2 * db + (my_col % 4) / 2) ^ S::swap(row);
                    const unsigned char *from = vbuf + row * S::kRow + piece * 16 + my_col % 2 * 8;
                    const u32x2 x = read_tr16(from), y = read_tr16(from + 16 * S::kRow);
                    v = u32x4{x.x, x.y, y.x, y.y};
                }
                return v;
            };
            if (S::kI8 || full) {
#pragma unroll
                for (int db = 0; db < S::kDims / 16; ++db)
#pragma unroll
                    for (int t = 0; t < KT / 32; ++t) {
                        const X8 v = __builtin_bit_cast(X8, values(db, t));
#pragma unroll
                        for (int i = 0; i < QT; ++i) o[i][db] = mma16(v, pr[i][t], o[i][db]);
                    }
            } else {
                // Values that a row does not see may be infinite or NaN, and zero times
                // those is no zero.
                X8 sight[QT][KT / 32];
#pragma unroll
                for (int i = 0; i < QT; ++i)
#pragma unroll
                    for (int e = 0; e < KT / 4; ++e)
                        sight[i][e / 8][e % 8] = (X)(((seen[i][e / 4] >> (e % 4)) & 1) ? 1.f : 0.f);
#pragma unroll
                for (int db = 0; db < S::kDims / 16; ++db) {
                    __builtin_amdgcn_sched_barrier(0);  // rare: no registers to work on several at once
#pragma unroll
                    for (int t = 0; t < KT / 32; ++t) {
                        const Parts<X> v(values(db, t));
#pragma unroll
                        for (int i = 0; i < QT; ++i) {
                            o[i][db] = mma16(v.finite, pr[i][t], o[i][db]);
                            const f32x4 up = mma16(v.up, sight[i][t], f32x4{0.f, 0.f, 0.f, 0.f});
                            const f32x4 down = mma16(v.down, sight[i][t], f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[i][db][e] += (up[e] > 0.f ? INFINITY : 0.f) - (down[e] > 0.f ? INFINITY : 0.f);
                        }
                    }
                }
            }
            __builtin_amdgcn_wave_barrier();
        }

        // the waves' parts meet: [wave][row][dim], then maximum and sum
        __syncthreads();
        float *const po = (float *)lds, *const pm = po + kWaves * 16 * QT * S::kOutPitch;
#pragma unroll
        for (int i = 0; i < QT; ++i) {
            float sum = l[i] + __shfl_xor(l[i], 16, 64);
            sum += __shfl_xor(sum, 32, 64);
            const int row = wave * 16 * QT + 16 * i + col;
            if (grp == 0) {
                if constexpr (S::kI8) pm[2 * row] = m[i] == kNoExponent ? -INFINITY : m[i];
                else pm[2 * row] = m[i] == -INFINITY ? -INFINITY : m[i] * qf[i];
                pm[2 * row + 1] = sum;
            }
            const float unit = S::kI8 ? __builtin_amdgcn_exp2f(mo[i] - m[i]) : 1.f;
#pragma unroll
            for (int db = 0; db < S::kDims / 16; ++db)
                *(f32x4 *)(po + row * S::kOutPitch + 16 * db + 4 * grp) = o[i][db] * unit;
        }
        __syncthreads();
        for (int e = (int)threadIdx.x; e < (r1 - r0) * S::kDims; e += kThreads) {
            const int row = e / S::kDims, d = e % S::kDims;
            if (d >= dim) continue;
            float top = pm[2 * row];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) top = fmaxf(top, pm[2 * (w * 16 * QT + row)]);
            float sum = 0.f, out = 0.f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const int at_row = w * 16 * QT + row;
                const float mw = pm[2 * at_row], f = mw == top ? 1.f : __builtin_amdgcn_exp2f(mw - top);
                sum += pm[2 * at_row + 1] * f;
                out += po[at_row * S::kOutPitch + d] * f;
            }
            if (n_chunks == 1) {
                Value<T>::store1((T *)a.out + out_line(p, seq, kvh, r0 + row) * dim + d, divide(out, sum));
            } else {
                const int64_t line = few_line(p, seq, kvh, r0 + row) * p.few.room + c;
                p.few.o[line * dim + d] = out;
                if (d == 0) p.few.ml[2 * line] = top, p.few.ml[2 * line + 1] = sum;
            }
        }
        __syncthreads();
    }
}

template <typename T, typename C> hipError_t launch2(const AttentionPlan &p, hipStream_t st) {
    const unsigned grid = (unsigned)(p.a.batch * p.few.chunks * p.a.cache.heads);
    const bool two = p.few.tile == 32;
    if (p.a.cache.dim <= 64) {
        if (two) attend_few<T, C, 1, 2><<<grid, kThreads, 0, st>>>(p);
        else attend_few<T, C, 1, 1><<<grid, kThreads, 0, st>>>(p);
    } else if (p.a.cache.dim <= 128) {
        if (two) attend_few<T, C, 2, 2><<<grid, kThreads, 0, st>>>(p);
        else attend_few<T, C, 2, 1><<<grid, kThreads, 0, st>>>(p);
    } else {
        attend_few<T, C, 4, 1><<<grid, kThreads, 0, st>>>(p);
    }
    return hipGetLastError();
}
template <typename T> hipError_t launch1(const AttentionPlan &p, hipStream_t st) {
    return p.a.cache.dtype == CBS_DTYPE_I8 ? launch2<T, int8_t>(p, st) : launch2<T, T>(p, st);
}

}  // namespace

hipError_t launch_attend_few(const AttentionPlan &p, hipStream_t st) {
    return p.a.dtype == CBS_DTYPE_BF16 ? launch1<__bf16>(p, st) : launch1<_Float16>(p, st);
}

}  // namespace cbs
