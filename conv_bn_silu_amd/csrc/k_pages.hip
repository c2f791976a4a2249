// k_pages.hip -- the pages of the paged cache by the sequences' lengths: room for new tokens
// with their slots and positions, and pages given back.
//
// Growing.  Where a sequence's tokens begin and which pages it takes are running sums over the
// sequences: one workgroup makes them (grow), a sequence a thread, 1024 at a time, and notes for each what
// its tokens need to know.  Where no sequence has more than a few new tokens, as in a decoding step, its
// thread goes on to write their slots and positions itself; else the tokens find their sequences by
// bisection, in the same workgroup where they are few, in a second kernel (place) where they are many.  Giving back
// is the same the other way round (release; count_back and move_back).
//
// Bound by latency: a launch, the lengths, two sums over the workgroup, a page of the stack.  64 sequences with a
// token each: 3.0 us on the GPU, and 2.8 to give them back (with the search for every token, and sums through LDS,
// 6.8 and 4.0); the two calls take the host 7.5.  1024 prompts, 2.1 million tokens: 4 and 9 us, given back 3 and 4 (16 MB, which a
// large copy would write in 3).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "b8_device.h"
#include "st_device.h"
#include "st_launch.h"

namespace cbs {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
// Up to so many sequences, tokens and entries of the table one workgroup does it all; so many tokens or
// pages of a sequence its thread does.  How many pages come back is not known before: giving back, us on the GPU, by one
// workgroup and by two launches (64 and 66 sequences of 1000 entries): a page each 2.7 and 5.0, 20 pages 4.6 and 5.2,
// 1000 pages 57 and 7.3; 300 sequences with 15 pages each 9.7 and 5.4.
constexpr int kFewSequences = kThreads, kFewTokens = 2048, kFewEntries = 65536, kOwn = 8;
constexpr int kFewItems = 4096;  // of release, that every workgroup sums by itself
constexpr uint32_t kManyTokens = 3u << 29;  // more than any batch has; twice that fits 32 bits
constexpr uint32_t kManyPages = INT32_MAX;  // as many as a pool may have; twice that fits, too

struct Grown {
    int len;    // tokens before, -1 where the sequence is left as it is
    int pages;  // of those
    int top;    // of the stack: its first new page's place
    int start;  // of its tokens in the batch
};

struct PagesParams {
    PagesArgs a;
    FastDiv page;
    bool whole;  // the one workgroup also writes slots
};

// Sums of `v` over the workgroup's threads before this one, which do not pass `most` (below 2^31); `all` gets that of
// all of them.  `part` is the workgroup's own, free when all threads have come here.
__device__ __forceinline__ uint32_t sum_before(uint32_t v, uint32_t most, uint32_t *part, uint32_t &all) {
    const int lane = (int)threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / 64);
    const uint32_t upto = lanes_upto(v, most), before = lane_from<0x138>(0, upto);  // the lane before's
    if (lane == 63) part[wave] = upto;
    __syncthreads();
    // the waves' sums, one to a lane of each 16
    uint32_t w = lane % 16 < (int)blockDim.x / 64 ? part[lane % 16] : 0;
    w = sixteen_upto(w, most);
    all = (uint32_t)__builtin_amdgcn_readlane((int)w, 15);
    const uint32_t waves = wave > 0 ? (uint32_t)__builtin_amdgcn_readlane((int)w, wave - 1) : 0;
    return min(before + waves, most);
}

__device__ __forceinline__ int pages_for(const FastDiv &page, int64_t tokens) {  // tokens < 2^31
    return (int)page.div((uint32_t)tokens) + (page.div((uint32_t)tokens) * page.d != (uint32_t)tokens);
}
// Page number `at` of a sequence: the table's, or the stack's where it is new.
__device__ __forceinline__ int page_at(const PagesArgs &a, int b, const Grown &g, int at) {
    return at < g.pages ? a.table[(int64_t)b * a.table_stride + at] : a.pool.free[g.top - (at - g.pages)];
}
__device__ __forceinline__ int slot_at(const PagesArgs &a, int page, int off) {
    return page >= 0 && page < a.pool.pages ? page * a.pool.page_size + off : -1;
}

// Of the sequences lo to hi, the last that begins at token t or before it (empty ones begin with the next).
__device__ __forceinline__ int sequence_of(const int32_t *starts, int t, int lo, int hi) {
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (starts[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Tokens [t, t + N) of the batch: their slots and positions, and the entries of new pages that begin with
// them.  Sequence b is the last that begins at t or before it, and none beyond `last` begins within them.
template <int N>
__device__ __forceinline__ void place_tokens(const PagesParams &p, int t, const int32_t *starts, const Grown *grown, int b, int last) {
    const PagesArgs &a = p.a;
    int slot[N], pos[N], page = -1, page_b = -1, page_no = -1;
    Grown g{-1, 0, 0, 0};
    int next = b < a.batch ? starts[b + 1] : t, had = -1;  // where b ends, and the sequence that g is of
#pragma unroll
    for (int i = 0; i < N; ++i) {
        slot[i] = -1, pos[i] = 0;
        if (t + i >= a.tokens) continue;
        if (b < a.batch && t + i >= next) {
            // the next one, or behind a run of idle ones
            if (++b < a.batch) next = starts[b + 1];
            if (b < a.batch && t + i >= next) {
                b = sequence_of(starts, t + i, b + 1, last);
                if (b < a.batch) next = starts[b + 1];
            }
        }
        if (b >= a.batch) continue;
        if (had != b) g = grown[b], had = b;
        if (g.len < 0) continue;
        pos[i] = g.len + (t + i - g.start);
        const int at = (int)p.page.div((uint32_t)pos[i]), off = pos[i] - at * (int)p.page.d;
        if (page_b != b || page_no != at) page = page_at(a, b, g, at), page_b = b, page_no = at;
        if (at >= g.pages && off == 0) a.table[(int64_t)b * a.table_stride + at] = page;
        slot[i] = slot_at(a, page, off);
    }
    if (N == 4 && t + 4 <= a.tokens) {
        ((Any16 *)(a.slots + t))->v = u32x4{(uint32_t)slot[0], (uint32_t)slot[1 % N], (uint32_t)slot[2 % N], (uint32_t)slot[3 % N]};
        ((Any16 *)(a.positions + t))->v = u32x4{(uint32_t)pos[0], (uint32_t)pos[1 % N], (uint32_t)pos[2 % N], (uint32_t)pos[3 % N]};
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (t + i < a.tokens) a.slots[t + i] = slot[i], a.positions[t + i] = pos[i];
    }
}

__global__ __launch_bounds__(kThreads) void grow(const PagesParams p) {
    __shared__ uint32_t part[2][kWaves];
    __shared__ int left_of[kWaves], taken_of[kWaves];
    __shared__ Grown few[kFewSequences];
    __shared__ int32_t few_starts[kFewSequences + 1];
    const PagesArgs &a = p.a;
    const int tid = (int)threadIdx.x, threads = (int)blockDim.x, lane = tid % 64, wave = tid / 64;
    const int count = max(0, min(a.pool.counts[0], (int)a.pool.pages));
    const int64_t room = a.table_width * a.pool.page_size;
    uint32_t tokens_before = 0, pages_before = 0;
    int left = 0, taken = 0;
    Grown g{-1, 0, 0, 0};
    int more = 0, start = 0, last_page = -1;
    for (int b0 = 0; b0 < a.batch; b0 += threads) {
        const int b = b0 + tid;
        const bool mine = b < a.batch;
        const int len = mine ? max(0, a.lens[b]) : 0;
        more = mine ? max(0, a.change[b]) : 0;
        // the page that the first new token may share with the last old one
        const int at = (int)p.page.div((uint32_t)len);
        if (p.whole && mine && at < a.table_width) last_page = a.table[(int64_t)b * a.table_stride + at];
        uint32_t all;
        const uint32_t begin = min(tokens_before + sum_before((uint32_t)more, kManyTokens, part[0], all), kManyTokens);
        const uint32_t end = min(begin + (uint32_t)more, kManyTokens);
        tokens_before = min(tokens_before + all, kManyTokens);
        const bool fits = more > 0 && end <= (uint32_t)a.tokens && (int64_t)len + more <= room && (int64_t)len + more <= INT32_MAX;
        const int had = pages_for(p.page, len), need = fits ? pages_for(p.page, (int64_t)len + more) - had : 0;
        const uint32_t pages = pages_before + sum_before((uint32_t)need, kManyTokens, part[1], all) + (uint32_t)need;
        pages_before += all;
        const bool grows = fits && pages <= (uint32_t)count;
        if (grows) taken = (int)pages;
        if (more > 0 && !grows) ++left;
        g = Grown{grows ? len : -1, had, count - 1 - ((int)pages - need), (int)begin};
        start = (int)min(begin, (uint32_t)a.tokens);
        if (mine) {
            a.starts[b] = start;
            if (grows) a.lens[b] = len + more;
            if (!p.whole) ((Grown *)a.workspace)[b] = g;
        }
        if (a.batch > threads) __syncthreads();  // part is free again
    }
    const int tokens_end = (int)min(tokens_before, (uint32_t)a.tokens);
    // what is summed over the workgroup at the end, on the way
    left = (int)team_sum_of<64>((uint32_t)left), taken = (int)team_max_of<64>((uint32_t)taken);
    if (lane == 0) left_of[wave] = left, taken_of[wave] = taken;
    const bool long_ones = __syncthreads_or(more > kOwn), own = p.whole && !long_ones;
    if (tid == 0) {
        a.starts[a.batch] = tokens_end;
        for (int w = 1; w < threads / 64; ++w) left += left_of[w], taken = max(taken, taken_of[w]);
        a.pool.counts[0] = count - taken;
        a.pool.counts[1] = max(0, (int)pages_before - count);
        a.pool.counts[2] = left;
    }
    if (!p.whole) return;
    if (own) {
        for (int i = 0; i < more; ++i) {
            const int t = start + i;
            if (t >= tokens_end) break;
            int slot = -1, pos = 0;
            if (g.len >= 0) {
                pos = g.len + i;
                const int at = (int)p.page.div((uint32_t)pos), off = pos - at * (int)p.page.d;
                const int page = at < g.pages ? last_page : a.pool.free[g.top - (at - g.pages)];
                if (at >= g.pages && off == 0) a.table[(int64_t)tid * a.table_stride + at] = page;
                slot = slot_at(a, page, off);
            }
            a.slots[t] = slot, a.positions[t] = pos;
        }
        for (int t = tokens_end + tid; t < a.tokens; t += threads) a.slots[t] = -1, a.positions[t] = 0;
        return;
    }
    if (tid < a.batch) few[tid] = g, few_starts[tid] = start;
    if (tid == 0) few_starts[a.batch] = tokens_end;
    __syncthreads();
    for (int t = tid; t < a.tokens; t += threads) place_tokens<1>(p, t, few_starts, few, sequence_of(few_starts, t, 0, a.batch), a.batch);
}

// 1024 tokens to a workgroup of 256.  Its first two waves look for the sequences of the first and the last of
// them, 64 ways at a time.  (All sequences into LDS at once, where there are few workgroups, took 0.4 us more.)
__global__ __launch_bounds__(256) void place(const PagesParams p) {
    __shared__ int ends[2];
    const PagesArgs &a = p.a;
    const int lane = (int)threadIdx.x % 64, wave = (int)threadIdx.x / 64, t0 = (int)blockIdx.x * 1024;
    if (wave < 2) {
        const int t = wave ? min(t0 + 1023, a.tokens - 1) : t0;
        int lo = 0, hi = a.batch;  // as in sequence_of
        while (lo < hi) {
            const int step = (hi - lo + 63) / 64, at = lo + (lane + 1) * step;
            const int upto = __builtin_popcountll(__ballot(at <= hi && a.starts[min(at, a.batch)] <= t));
            const int now = min(hi, lo + (upto + 1) * step - 1);
            lo += upto * step;
            hi = now;
        }
        if (lane == 0) ends[wave] = lo;
    }
    __syncthreads();
    const int t = t0 + (int)threadIdx.x * 4;
    if (t < a.tokens) place_tokens<4>(p, t, a.starts, (const Grown *)a.workspace, sequence_of(a.starts, t, ends[0], ends[1]), ends[1]);
}

// Giving back.  Only entries that name pages of the pool go to the stack: in a row there may be holes (pages
// that a window has left behind).  So an entry's place is the number of such entries after it, above what the stack
// holds, and the sums run from the last entry to the first.
__device__ __forceinline__ bool in_pool(const PagesArgs &a, int page) { return page >= 0 && page < a.pool.pages; }
__device__ __forceinline__ void push(const PagesArgs &a, int64_t to, int page) {
    if (to < a.pool.pages) a.pool.free[to] = page;
}
struct Cut {
    int held, keep;    // tokens as the lengths have them, and that stay
    int first, count;  // entries of its row that go
};
__device__ __forceinline__ Cut cut_of(const PagesParams &p, int b) {
    const int held = p.a.lens[b], len = max(0, held), keep = min(len, max(0, p.a.change[b])), first = pages_for(p.page, keep);
    return Cut{held, keep, first, max(0, (int)min((int64_t)pages_for(p.page, len), p.a.table_width) - first)};
}

// All of it by one workgroup, a sequence a thread.
__global__ __launch_bounds__(kThreads) void release(const PagesParams p) {
    __shared__ uint32_t part[kWaves], of_64[2][4 * kWaves];
    __shared__ int few_first[kFewSequences];
    __shared__ int32_t few_begin[kFewSequences];  // entries of those before
    const PagesArgs &a = p.a;
    const int tid = (int)threadIdx.x, threads = (int)blockDim.x;
    const int count = max(0, min(a.pool.counts[0], (int)a.pool.pages));
    const bool mine = tid < a.batch;
    const Cut c = mine ? cut_of(p, tid) : Cut{0, 0, 0, 0};
    int32_t *const row = a.table + (int64_t)tid * a.table_stride + c.first;
    if (c.keep != c.held) a.lens[tid] = c.keep;
    // its own entries, if they are few, on their way
    int page[kOwn];
    uint32_t there = 0;  // a bit for each page of the pool
#pragma unroll
    for (int i = 0; i < kOwn; ++i) page[i] = i < c.count ? row[i] : -1;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) there |= in_pool(a, page[i]) ? 1u << i : 0;
    uint32_t all;
    int64_t base = count;
    if (!__syncthreads_or(c.count > kOwn)) {  // and everyone has read the count
        const uint32_t before = sum_before((uint32_t)__builtin_popcount(there), kManyPages, part, all);
        int64_t to = base + all - 1 - before;
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
            if (i >= c.count) break;
            if (there >> i & 1) push(a, to--, page[i]);
            row[i] = -1;
        }
        base += all;
    } else {
        // entries over the threads, from the last, four on their way at a time: of each 64 those of the pool are
        // counted, and the counts summed by every wave
        uint32_t entries;
        const uint32_t begin = sum_before((uint32_t)c.count, kManyPages, part, entries);
        few_first[tid] = c.first, few_begin[tid] = (int)begin;
        __syncthreads();
        const int lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64), waves = threads / 64;
        int turn = 0;
        for (int e0 = (int)entries - 1 - tid; e0 + tid >= 0; e0 -= 4 * threads, turn ^= 1) {
            int32_t *entry[4];
            int page[4];
            uint64_t those[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int e = e0 - u * threads;
                page[u] = -1;
                if (e < 0) continue;
                const int b = sequence_of(few_begin, e, 0, a.batch - 1);
                entry[u] = a.table + (int64_t)b * a.table_stride + few_first[b] + (e - few_begin[b]);
                page[u] = *entry[u];
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                those[u] = __ballot(in_pool(a, page[u]));
                if (lane == 0) of_64[turn][u * kWaves + wave] = (uint32_t)__builtin_popcountll(those[u]);
            }
            __syncthreads();
            const uint32_t upto = lanes_upto(lane % kWaves < waves ? of_64[turn][lane] : 0, kManyPages);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int its = u * kWaves + wave;
                const uint32_t before = its ? (uint32_t)__builtin_amdgcn_readlane((int)upto, its - 1) : 0;
                if (those[u] >> lane & 1) push(a, base + before + __builtin_popcountll(those[u] & ((1ull << lane) - 1)), page[u]);
                if (e0 - u * threads >= 0) *entry[u] = -1;
            }
            base += (uint32_t)__builtin_amdgcn_readlane((int)upto, 63);
        }
    }
    if (tid == 0) a.pool.counts[0] = (int)min(base, a.pool.pages);
}

// Where one workgroup would take long: items, each a part of a sequence's entries; `parts` of them to a sequence, in
// the order of the entries.  count_back notes what each has, move_back moves it.
struct Back {
    int first, count;  // entries of the row
    int there;         // of them pages of the pool
    int after;         // such entries of all items after it; where there are many, by sum_back
};
struct BackPlan {
    Back *items;
    int32_t *there, *count;  // the items' once more, side by side; the stack's before
    int n, parts;
};

// An item to a wave.
__global__ __launch_bounds__(64) void count_back(const PagesParams p, const BackPlan plan) {
    const PagesArgs &a = p.a;
    const int lane = (int)threadIdx.x, i = (int)blockIdx.x, b = i / plan.parts;
    const Cut c = cut_of(p, b);
    const int64_t share = ((int64_t)c.count + plan.parts - 1) / plan.parts, from = min(share * (i - b * plan.parts), (int64_t)c.count);
    const int first = c.first + (int)from, n = (int)min(share, c.count - from);
    const int32_t *const row = a.table + (int64_t)b * a.table_stride + first;
    uint32_t there = 0;
    for (int64_t e0 = 0; e0 < n; e0 += 256) {
        int page[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) page[u] = e0 + u * 64 + lane < n ? row[e0 + u * 64 + lane] : -1;
#pragma unroll
        for (int u = 0; u < 4; ++u) there += in_pool(a, page[u]);
    }
    there = team_sum_of<64>(there);
    if (lane != 0) return;
    plan.items[i] = Back{first, n, (int)there, 0};
    plan.there[i] = (int)there;
    if (i == 0) *plan.count = max(0, min(a.pool.counts[0], (int)a.pool.pages));
}

// Where there are more items than a workgroup of move_back sums by itself.
__global__ __launch_bounds__(kThreads) void sum_back(const BackPlan plan) {
    __shared__ uint32_t part[2][kWaves];
    uint32_t after = 0, all;
    int turn = 0;
    for (int i0 = plan.n - 1; i0 >= 0; i0 -= kThreads, turn ^= 1) {
        const int i = i0 - (int)threadIdx.x;
        const uint32_t before = sum_before(i >= 0 ? (uint32_t)plan.there[i] : 0, kManyPages, part[turn], all);
        if (i >= 0) plan.items[i].after = (int)min(after + before, kManyPages);
        after = min(after + all, kManyPages);
    }
}

__global__ __launch_bounds__(256) void move_back(const PagesParams p, const BackPlan plan) {
    __shared__ double sums[4];
    __shared__ int part[2][4];
    const PagesArgs &a = p.a;
    const int tid = (int)threadIdx.x, lane = tid % 64, wave = tid / 64, i = (int)blockIdx.x, b = i / plan.parts;
    const Back r = plan.items[i];
    int32_t *const row = a.table + (int64_t)b * a.table_stride + r.first;
    int next = tid < r.count ? row[r.count - 1 - tid] : -1;  // on its way while the others' are summed
    if (tid == 0 && i == b * plan.parts) {
        const Cut c = cut_of(p, b);  // no other workgroup reads the lengths any more
        if (c.keep != c.held) a.lens[b] = c.keep;
    }
    if (r.count == 0 && i != 0) return;
    int64_t base = *plan.count;
    if (plan.n <= kFewItems) {
        double after = 0;  // whole numbers below 2^53
        for (int j = i + 1 + tid; j < plan.n; j += 256) after += plan.there[j];
        after = team_sum<64>(after);
        if (lane == 0) sums[wave] = after;
        __syncthreads();
        base += (int64_t)(sums[0] + sums[1] + sums[2] + sums[3]);
    } else {
        base += r.after;
    }
    if (tid == 0 && i == 0) a.pool.counts[0] = (int)min(base + r.there, a.pool.pages);
    const bool holes = r.there != r.count;
    int turn = 0;
    for (int64_t e = (int64_t)r.count - 1 - tid; e + tid >= 0; e -= 256, turn ^= 1) {
        const int page = next;
        if (e >= 256) next = row[e - 256];
        bool there = e >= 0;
        int before = tid, all = 256;
        if (holes) {
            there = there && in_pool(a, page);
            const uint64_t those = __ballot(there);
            if (lane == 0) part[turn][wave] = __builtin_popcountll(those);
            __syncthreads();
            before = __builtin_popcountll(those & ((1ull << lane) - 1)), all = 0;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                if (w < wave) before += part[turn][w];
                all += part[turn][w];
            }
        }
        if (there) push(a, base + before, page);
        if (e >= 0) row[e] = -1;
        base += all;
    }
}

bool grows_whole(int64_t batch, int64_t tokens) { return batch <= kFewSequences && tokens <= kFewTokens; }
bool releases_whole(int64_t batch, int64_t width) { return batch <= kFewSequences && batch * width <= kFewEntries; }
// Items to a sequence: each has the better part of 1024 entries or more, and a few sequences make no more items than
// move_back sums.
int64_t parts_of(int64_t batch, int64_t width) {
    return std::max<int64_t>(1, std::min<int64_t>((width + 1023) / 1024, kFewItems / batch));
}
// Whole waves for n sequences or tokens.
int threads_for(int64_t n) { return (int)std::min<int64_t>(kThreads, std::max<int64_t>(64, (n + 63) / 64 * 64)); }

}  // namespace

int64_t grow_workspace(int64_t batch, int64_t tokens) { return grows_whole(batch, tokens) ? 0 : batch * (int64_t)sizeof(Grown); }
int64_t release_workspace(int64_t batch, int64_t width) {
    return releases_whole(batch, width) ? 0 : batch * parts_of(batch, width) * (int64_t)(sizeof(Back) + 4) + 4;
}

hipError_t launch_grow_pages(const PagesArgs &a, hipStream_t st) {
    const PagesParams p{a, make_fastdiv((uint32_t)a.pool.page_size), grows_whole(a.batch, a.tokens)};
    grow<<<1, threads_for(p.whole ? std::max(a.batch, a.tokens) : a.batch), 0, st>>>(p);
    if (!p.whole && a.tokens > 0) place<<<(unsigned)(((int64_t)a.tokens + 1023) / 1024), 256, 0, st>>>(p);
    return hipGetLastError();
}

hipError_t launch_release_pages(const PagesArgs &a, hipStream_t st) {
    const bool whole = releases_whole(a.batch, a.table_width);
    const PagesParams p{a, make_fastdiv((uint32_t)a.pool.page_size), whole};
    if (whole) {
        release<<<1, threads_for(std::max<int64_t>(a.batch, a.batch * a.table_width / 16)), 0, st>>>(p);
        return hipGetLastError();
    }
    const int parts = (int)parts_of(a.batch, a.table_width), n = a.batch * parts;
    Back *const items = (Back *)a.workspace;
    int32_t *const there = (int32_t *)(items + n);
    const BackPlan plan{items, there, there + n, n, parts};
    count_back<<<(unsigned)n, 64, 0, st>>>(p, plan);
    if (n > kFewItems) sum_back<<<1, kThreads, 0, st>>>(plan);
    move_back<<<(unsigned)n, 256, 0, st>>>(p, plan);
    return hipGetLastError();
}

}  // namespace cbs
