// k_pages.hip -- the pages of the paged cache by the sequences' lengths: room for new tokens
// with their slots and positions, and pages given back.
//
// Growing.  Where a sequence's tokens begin and which pages it takes are running sums over the
// sequences: one workgroup makes them (grow), a sequence a thread, 1024 at a time, and notes for each what
// its tokens need to know.  Where no sequence has more than a few new tokens, as in a decoding step, its
// thread goes on to write their slots and positions itself; else the tokens find their sequences by
// bisection, in the same workgroup where they are few, in a second kernel (place) where they are many.  Giving back
// is the same the other way round (release, move_back).
//
// Bound by latency: a launch, the lengths, two sums over the workgroup, a page of the stack.  64 sequences with a
// token each: 3.0 us on the GPU, and 2.7 to give them back (with the search for every token, and sums through LDS,
// 6.8 and 4.0); the two calls take the host 7.5.  1024 prompts, 2.1 million tokens: 4 and 9 us, given back 3 and 3 (16 MB, which a
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
// pages of a sequence its thread does.  How many pages come back is not known before: growing and giving back, us, by one
// workgroup and by two launches, 64 sequences of 1001 entries: a page each 8.2 and 11.5, 20 pages 11.9 and 17.5, 1000 pages
// 60 and 18.
constexpr int kFewSequences = kThreads, kFewTokens = 2048, kFewEntries = 65536, kOwn = 8;
constexpr uint32_t kManyTokens = 3u << 29;  // more than any batch has; twice that fits 32 bits
constexpr uint32_t kManyPages = INT32_MAX;  // as many as a pool may have; twice that fits, too

struct Grown {
    int len;    // tokens before, -1 where the sequence is left as it is
    int pages;  // of those
    int top;    // of the stack: its first new page's place
    int start;  // of its tokens in the batch
};
struct Released {
    int first, count;  // entries of its row
    int top;           // of the stack: the first's place
    int pad;
};

struct PagesParams {
    PagesArgs a;
    FastDiv page;
    bool whole;  // the one workgroup also writes slots, or moves pages
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
// them.  Sequence b is the last that begins at t or before it.
template <int N>
__device__ __forceinline__ void place_tokens(const PagesParams &p, int t, const int32_t *starts, const Grown *grown, int b) {
    const PagesArgs &a = p.a;
    int slot[N], pos[N], page = -1, page_b = -1, page_no = -1;
    Grown g{-1, 0, 0, 0};
    int next = t, had = -1;  // where b ends, and the sequence that g is of
#pragma unroll
    for (int i = 0; i < N; ++i) {
        slot[i] = -1, pos[i] = 0;
        while (b < a.batch && t + i >= next) {
            next = starts[b + 1];
            if (t + i >= next) ++b;
        }
        if (b >= a.batch || t + i >= a.tokens) continue;
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
    for (int t = tid; t < a.tokens; t += threads) place_tokens<1>(p, t, few_starts, few, sequence_of(few_starts, t, 0, a.batch));
}

// 1024 tokens to a workgroup of 256.  Its first two waves look for the sequences of the first and the last of
// them, 64 ways at a time.  (All sequences into LDS at once, where there are few workgroups: 6.8 us, so 6.4.)
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
    if (t < a.tokens) place_tokens<4>(p, t, a.starts, (const Grown *)a.workspace, sequence_of(a.starts, t, ends[0], ends[1]));
}

// Entries [from, from + step, ...) of a sequence's pages that go back.
__device__ __forceinline__ void give_back(const PagesArgs &a, int b, const Released &r, int from, int step) {
    int32_t *const row = a.table + (int64_t)b * a.table_stride + r.first;
    for (int i = from; i < r.count; i += step) {
        const int page = row[i], to = r.top - i;
        if (to >= 0 && to < a.pool.pages) a.pool.free[to] = page;
        row[i] = -1;
    }
}

__global__ __launch_bounds__(kThreads) void release(const PagesParams p) {
    __shared__ uint32_t part[kWaves];
    __shared__ Released few[kFewSequences];
    __shared__ int32_t few_begin[kFewSequences];  // pages that those before give back
    const PagesArgs &a = p.a;
    const int tid = (int)threadIdx.x, threads = (int)blockDim.x;
    const int count = max(0, min(a.pool.counts[0], (int)a.pool.pages));
    uint32_t total = 0;
    Released r{0, 0, 0, 0};
    // The first page given back lies on top of all, so that their number comes first: twice through the
    // sequences, or once where each has a thread.
    for (int pass = a.batch <= threads ? 1 : 0; pass < 2; ++pass) {
        uint32_t before = 0;
        for (int b0 = 0; b0 < a.batch; b0 += threads) {
            const int b = b0 + tid;
            const bool mine = b < a.batch;
            const int held = mine ? a.lens[b] : 0, len = max(0, held), keep = mine ? min(len, max(0, a.change[b])) : 0;
            const int first = pages_for(p.page, keep);
            const int last = (int)min((int64_t)pages_for(p.page, len), a.table_width);
            const int n = max(0, last - first);
            uint32_t all;
            const uint32_t upto = before + sum_before((uint32_t)n, kManyPages, part, all);
            before = min(before + all, kManyPages);
            if (a.batch <= threads) total = all;
            if (pass == 1 && mine) {
                const int64_t top = (int64_t)count + total - 1 - upto;
                r = Released{first, n, (int)min(top, (int64_t)INT32_MAX), 0};
                if (keep != held) a.lens[b] = keep;
                if (!p.whole) ((Released *)a.workspace)[b] = r;
            }
            if (a.batch > threads) __syncthreads();  // part is free again
        }
        total = before;
    }
    if (!__syncthreads_or(p.whole && r.count > kOwn)) {  // and everyone has read the count
        if (p.whole && r.count > 0) give_back(a, tid, r, 0, 1);
    } else {
        // pages over the threads, four on their way at a time
        few[tid] = r;
        few_begin[tid] = count + (int)total - 1 - r.top;
        __syncthreads();
        for (int e0 = tid; e0 < (int)total; e0 += 4 * threads) {
            int32_t *entry[4];
            int page[4], to[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int e = e0 + u * threads;
                if (e >= (int)total) continue;
                const int b = sequence_of(few_begin, e, 0, a.batch - 1), i = e - few_begin[b];
                entry[u] = a.table + (int64_t)b * a.table_stride + few[b].first + i;
                page[u] = *entry[u], to[u] = few[b].top - i;
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (e0 + u * threads >= (int)total) continue;
                if (to[u] >= 0 && to[u] < a.pool.pages) a.pool.free[to[u]] = page[u];
                *entry[u] = -1;
            }
        }
    }
    if (tid == 0) a.pool.counts[0] = (int)min((int64_t)count + total, a.pool.pages);
}

// A part of a sequence's pages to a workgroup: blockIdx.x the sequence, blockIdx.y the part.
__global__ __launch_bounds__(256) void move_back(const PagesParams p) {
    const int b = (int)blockIdx.x;
    const Released r = ((const Released *)p.a.workspace)[b];
    give_back(p.a, b, r, (int)blockIdx.y * 256 + (int)threadIdx.x, (int)gridDim.y * 256);
}

bool grows_whole(int64_t batch, int64_t tokens) { return batch <= kFewSequences && tokens <= kFewTokens; }
bool releases_whole(int64_t batch, int64_t width) { return batch <= kFewSequences && batch * width <= kFewEntries; }
// Whole waves for n sequences or tokens.
int threads_for(int64_t n) { return (int)std::min<int64_t>(kThreads, std::max<int64_t>(64, (n + 63) / 64 * 64)); }

}  // namespace

int64_t grow_workspace(int64_t batch, int64_t tokens) { return grows_whole(batch, tokens) ? 0 : batch * (int64_t)sizeof(Grown); }
int64_t release_workspace(int64_t batch, int64_t width) {
    return releases_whole(batch, width) ? 0 : batch * (int64_t)sizeof(Released);
}

hipError_t launch_grow_pages(const PagesArgs &a, hipStream_t st) {
    const PagesParams p{a, make_fastdiv((uint32_t)a.pool.page_size), grows_whole(a.batch, a.tokens)};
    grow<<<1, threads_for(p.whole ? std::max(a.batch, a.tokens) : a.batch), 0, st>>>(p);
    if (!p.whole && a.tokens > 0) place<<<(unsigned)(((int64_t)a.tokens + 1023) / 1024), 256, 0, st>>>(p);
    return hipGetLastError();
}

hipError_t launch_release_pages(const PagesArgs &a, hipStream_t st) {
    const PagesParams p{a, make_fastdiv((uint32_t)a.pool.page_size), releases_whole(a.batch, a.table_width)};
    release<<<1, threads_for(p.whole ? std::max<int64_t>(a.batch, a.batch * a.table_width / 16) : a.batch), 0, st>>>(p);
    if (!p.whole) {
        const int64_t parts = std::max<int64_t>(1, std::min<int64_t>((a.table_width + 1023) / 1024, 16384 / a.batch));
        move_back<<<dim3((unsigned)a.batch, (unsigned)parts), 256, 0, st>>>(p);
    }
    return hipGetLastError();
}

}  // namespace cbs
