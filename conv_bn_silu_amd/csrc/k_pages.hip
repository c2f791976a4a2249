// k_pages.hip -- the pages of the paged cache by the sequences' lengths: room for new tokens
// with their slots and positions, and pages given back.
//
// Growing.  Where a sequence's tokens begin and which pages it takes are running sums over the
// sequences: one workgroup makes them (grow), 1024 sequences at a time, and notes for each what
// its tokens need to know.  The tokens then find their sequences by bisection and write a
// slot and a position each, and the table's entry where a page begins: the same workgroup
// where they are few, else a second kernel (place).  Giving back is the same the other way round.
//
// Bound by latency for a step's single tokens, by HBM (8 bytes a token) for prompts.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "b8_device.h"
#include "st_launch.h"

namespace cbs {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
// Up to so many sequences and tokens (pages of the table) one workgroup does it all.
constexpr int kFewSequences = kThreads, kFewTokens = 8192, kFewEntries = 65536;
constexpr uint32_t kManyTokens = 3u << 29;  // more than any batch has; twice that fits 32 bits

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
    const int lane = (int)threadIdx.x % 64, wave = (int)threadIdx.x / 64;
    v = min(v, most);
#pragma unroll
    for (int o = 1; o < 64; o *= 2) {
        const uint32_t x = (uint32_t)__shfl_up((int)v, o, 64);
        if (lane >= o) v = min(v + x, most);
    }
    if (lane == 63) part[wave] = v;
    __syncthreads();
    uint32_t before = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        if (w == wave) before = sum;
        sum = min(sum + part[w], most);
    }
    all = sum;
    const uint32_t x = (uint32_t)__shfl_up((int)v, 1, 64);
    return lane == 0 ? before : min(before + x, most);
}

__device__ __forceinline__ int pages_for(const FastDiv &page, int64_t tokens) {  // tokens < 2^31
    return (int)page.div((uint32_t)tokens) + (page.div((uint32_t)tokens) * page.d != (uint32_t)tokens);
}

// Tokens [t, t + 4) of the batch: their slots and positions, and the entries of pages that begin with
// them.  starts and grown of all sequences; sequence lo or one after it has token t.
__device__ __forceinline__ void place4(const PagesParams &p, int t, const int32_t *starts, const Grown *grown, int lo, int hi) {
    const PagesArgs &a = p.a;
    // the last sequence that begins at t or before it: empty ones have the same start as the next
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (starts[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    int slot[4], pos[4];
    int b = lo;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        slot[i] = -1, pos[i] = 0;
        while (b < a.batch && t + i >= starts[b + 1]) ++b;
        if (b >= a.batch || t + i >= a.tokens) continue;
        const Grown g = grown[b];
        if (g.len < 0) continue;
        pos[i] = g.len + (t + i - g.start);
        const int at = (int)p.page.div((uint32_t)pos[i]), off = pos[i] - at * (int)p.page.d;
        int32_t *const entry = a.table + (int64_t)b * a.table_stride + at;
        const int page = at < g.pages ? *entry : a.pool.free[g.top - (at - g.pages)];
        if (at >= g.pages && off == 0) *entry = page;
        if (page >= 0 && page < a.pool.pages) slot[i] = page * (int)p.page.d + off;
    }
    if (t + 4 <= a.tokens) {
        ((Any16 *)(a.slots + t))->v = u32x4{(uint32_t)slot[0], (uint32_t)slot[1], (uint32_t)slot[2], (uint32_t)slot[3]};
        ((Any16 *)(a.positions + t))->v = u32x4{(uint32_t)pos[0], (uint32_t)pos[1], (uint32_t)pos[2], (uint32_t)pos[3]};
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (t + i < a.tokens) a.slots[t + i] = slot[i], a.positions[t + i] = pos[i];
    }
}

__global__ __launch_bounds__(kThreads) void grow(const PagesParams p) {
    __shared__ uint32_t part[2][kWaves];
    __shared__ int left_of[kWaves], last_of[kWaves];
    __shared__ Grown few[kFewSequences];
    __shared__ int32_t few_starts[kFewSequences + 1];
    const PagesArgs &a = p.a;
    const int tid = (int)threadIdx.x, lane = tid % 64, wave = tid / 64;
    const int count = max(0, min(a.pool.counts[0], (int)a.pool.pages));
    const int64_t room = a.table_width * a.pool.page_size;
    uint32_t tokens_before = 0, pages_before = 0;
    int left = 0, taken = 0;
    for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
        const int b = b0 + tid;
        const bool mine = b < a.batch;
        const int len = mine ? max(0, a.lens[b]) : 0, more = mine ? max(0, a.change[b]) : 0;
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
        const Grown g{grows ? len : -1, had, count - 1 - ((int)pages - need), (int)begin};
        const int start = (int)min(begin, (uint32_t)a.tokens);
        if (mine) {
            a.starts[b] = start;
            if (grows) a.lens[b] = len + more;
            if (p.whole) few[b] = g, few_starts[b] = start;
            else ((Grown *)a.workspace)[b] = g;
        }
        __syncthreads();  // part is free again
    }
#pragma unroll
    for (int o = 1; o < 64; o *= 2) {
        left += __shfl_xor(left, o, 64);
        taken = max(taken, __shfl_xor(taken, o, 64));
    }
    if (lane == 0) left_of[wave] = left, last_of[wave] = taken;
    __syncthreads();
    if (tid == 0) {
        const int end = (int)min(tokens_before, (uint32_t)a.tokens);
        a.starts[a.batch] = end;
        if (p.whole) few_starts[a.batch] = end;
        for (int w = 1; w < kWaves; ++w) left += left_of[w], taken = max(taken, last_of[w]);
        a.pool.counts[0] = count - taken;
        a.pool.counts[1] = max(0, (int)pages_before - count);
        a.pool.counts[2] = left;
    }
    if (!p.whole) return;
    __syncthreads();
    for (int t = 4 * tid; t < a.tokens; t += 4 * kThreads) place4(p, t, few_starts, few, 0, a.batch);
}

// 1024 tokens to a workgroup of 256.
__global__ __launch_bounds__(256) void place(const PagesParams p) {
    const PagesArgs &a = p.a;
    const int t = ((int)blockIdx.x * 256 + (int)threadIdx.x) * 4;
    if (t < a.tokens) place4(p, t, a.starts, (const Grown *)a.workspace, 0, a.batch);
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
    const PagesArgs &a = p.a;
    const int tid = (int)threadIdx.x;
    const int count = max(0, min(a.pool.counts[0], (int)a.pool.pages));
    // twice: the first page given back lies on top of all, so that their number comes first
    uint32_t total = 0;
    for (int pass = 0; pass < 2; ++pass) {
        uint32_t before = 0;
        for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
            const int b = b0 + tid;
            const bool mine = b < a.batch;
            const int len = mine ? max(0, a.lens[b]) : 0, keep = mine ? min(len, max(0, a.change[b])) : 0;
            const int first = pages_for(p.page, keep);
            const int last = (int)min((int64_t)pages_for(p.page, len), a.table_width);
            const int n = max(0, last - first);
            uint32_t all;
            const uint32_t upto = before + sum_before((uint32_t)n, kManyTokens, part, all);
            if (pass == 1 && mine) {
                const int64_t top = (int64_t)count + total - 1 - upto;
                const Released r{first, n, (int)min(top, (int64_t)INT32_MAX), 0};
                if (keep < len) a.lens[b] = keep;
                if (p.whole) few[b] = r;
                else ((Released *)a.workspace)[b] = r;
            }
            before = min(before + all, kManyTokens);
            __syncthreads();
        }
        total = before;
    }
    if (tid == 0) a.pool.counts[0] = (int)min((int64_t)count + total, a.pool.pages);
    if (!p.whole) return;
    for (int b = tid / 64; b < a.batch; b += kWaves) give_back(a, b, few[b], tid % 64, 64);
}

// A part of a sequence's pages to a workgroup: blockIdx.x the sequence, blockIdx.y the part.
__global__ __launch_bounds__(256) void move_back(const PagesParams p) {
    const int b = (int)blockIdx.x;
    const Released r = ((const Released *)p.a.workspace)[b];
    give_back(p.a, b, r, (int)blockIdx.y * 256 + (int)threadIdx.x, (int)gridDim.y * 256);
}

bool grows_whole(int64_t batch, int64_t tokens) { return batch <= kFewSequences && tokens <= kFewTokens; }
bool releases_whole(int64_t batch, int64_t width) { return batch <= kFewSequences && batch * width <= kFewEntries; }

}  // namespace

int64_t grow_workspace(int64_t batch, int64_t tokens) { return grows_whole(batch, tokens) ? 0 : batch * (int64_t)sizeof(Grown); }
int64_t release_workspace(int64_t batch, int64_t width) {
    return releases_whole(batch, width) ? 0 : batch * (int64_t)sizeof(Released);
}

hipError_t launch_grow_pages(const PagesArgs &a, hipStream_t st) {
    const PagesParams p{a, make_fastdiv((uint32_t)a.pool.page_size), grows_whole(a.batch, a.tokens)};
    grow<<<1, kThreads, 0, st>>>(p);
    if (!p.whole && a.tokens > 0) place<<<(unsigned)(((int64_t)a.tokens + 1023) / 1024), 256, 0, st>>>(p);
    return hipGetLastError();
}

hipError_t launch_release_pages(const PagesArgs &a, hipStream_t st) {
    const PagesParams p{a, make_fastdiv((uint32_t)a.pool.page_size), releases_whole(a.batch, a.table_width)};
    release<<<1, kThreads, 0, st>>>(p);
    if (!p.whole) {
        const int64_t parts = std::max<int64_t>(1, std::min<int64_t>((a.table_width + 1023) / 1024, 16384 / a.batch));
        move_back<<<dim3((unsigned)a.batch, (unsigned)parts), 256, 0, st>>>(p);
    }
    return hipGetLastError();
}

}  // namespace cbs
