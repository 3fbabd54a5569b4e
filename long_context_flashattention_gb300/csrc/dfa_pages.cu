// dfa_pages.cu -- the pages behind a paged cache: sequences forked, pages taken for rows
// to come, copied and given back; and the rows of a cache that are kept moved together.
//
// A pool is its table, the pages that each sequence holds and a count of holders per
// page.  There is no list of free pages: a page that nobody holds is free, and the
// lowest ones are taken first, so that what a call gives depends on the pool's state
// alone.
#include "dfa_branch.h"
#include "dfa_serve.cuh"

namespace dfa {

namespace {

// Sites of DFA_ERR_BOUNDS in DevStatus::where.
constexpr int kSiteKept = 104, kSiteHeld = 105, kSiteSource = 106, kSitePool = 107,
              kSiteRefs = 108;

__device__ __forceinline__ bool pool_page(const PoolView& p, int32_t b, int32_t id)
{
    if (id >= 0 && id < p.npages)
        return true;
    cache_fault(p.status, kSitePage, b);
    return false;
}

// Pages that sequence b holds; false (and reported): not a number of pages.
__device__ __forceinline__ bool pages_held(const PoolView& p, int32_t b, int32_t& held)
{
    held = p.held[b];
    if (held >= 0 && held <= p.max_pages)
        return true;
    cache_fault(p.status, kSiteHeld, b);
    return false;
}

// (A page without holders keeps its count: at -1 it would not be free, and with its next
// holder it would.)
__device__ __forceinline__ void release(const PoolView& p, int32_t b, int32_t id)
{
    if (pool_page(p, b, id) && atomicSub(p.refs + id, 1) <= 0) {
        atomicAdd(p.refs + id, 1);
        cache_fault(p.status, kSiteRefs, b);
    }
}

// ---------------------------------------------------------------------------
// fork: what the sequences will hold, gathered before anything changes; then taken over
// ---------------------------------------------------------------------------
// What sequence b will hold: entries i, i + step, ..
__device__ __forceinline__ void fork_gather(const ForkParams& p, int32_t b, int32_t i, int32_t step)
{
    const int32_t src = p.src[b];
    if (src == b)
        return;
    int32_t held = 0, len = 0;
    bool ok = src >= -1 && src < p.p.B;
    if (!ok)
        cache_fault(p.p.status, kSiteSource, b);
    else if (src >= 0) {
        ok = pages_held(p.p, src, held);
        len = p.p.seq_lens[src];
        if (len < 0 || len > (int64_t)p.p.max_pages << p.p.page_log2) {
            cache_fault(p.p.status, kSiteSeqLen, src);
            ok = false;
        }
    }
    if (i == 0) {
        p.held[b] = ok ? held : -1;  // -1: stays as it is
        p.lens[b] = len;
    }
    if (!ok)
        return;
    const int32_t* from = p.p.table + (int64_t)src * p.p.max_pages;
    int32_t* to = p.rows + (int64_t)b * p.p.max_pages;
    for (int32_t e = i; e < held; e += step)
        to[e] = from[e];
}

// (Entries that stay, the shared beginning of beams for one, cost no atomics.)  Returns
// whether `held` and `len` are b's from now on, which is to be written when all have read
// what it held.
__device__ __forceinline__ bool fork_apply(const ForkParams& p, int32_t b, int32_t i, int32_t step)
{
    if (p.src[b] == b)
        return false;
    const int32_t held = p.held[b];
    int32_t old_held;
    if (held < 0 || !pages_held(p.p, b, old_held))
        return false;
    int32_t* row = p.p.table + (int64_t)b * p.p.max_pages;
    const int32_t* from = p.rows + (int64_t)b * p.p.max_pages;
    const int32_t end = max(held, old_held);
    for (int32_t e = i; e < end; e += step) {
        const int32_t was = e < old_held ? row[e] : -1, now = e < held ? from[e] : -1;
        if (was == now && e < old_held && e < held)
            continue;
        if (e < held) {
            row[e] = now;
            if (pool_page(p.p, b, now))
                atomicAdd(p.p.refs + now, 1);
        }
        if (e < old_held)
            release(p.p, b, was);
    }
    return true;
}

__device__ __forceinline__ void fork_end(const ForkParams& p, int32_t b)
{
    p.p.held[b] = p.held[b];
    p.p.seq_lens[b] = p.lens[b];
}

__global__ void __launch_bounds__(256) fork_gather_kernel(const __grid_constant__ ForkParams p)
{
    fork_gather(p, blockIdx.x, blockIdx.y * blockDim.x + threadIdx.x, gridDim.y * blockDim.x);
}

__global__ void __launch_bounds__(256) fork_apply_kernel(const __grid_constant__ ForkParams p)
{
    const bool taken = fork_apply(p, blockIdx.x, threadIdx.x, blockDim.x);
    __syncthreads();
    if (taken && threadIdx.x == 0)
        fork_end(p, blockIdx.x);
}

// Both for a few sequences, a warp each, in one launch (8 beams: 4.4 -> 3.5 us).
constexpr int kForkHere = 32;

__global__ void __launch_bounds__(32 * kForkHere) fork_kernel(const __grid_constant__ ForkParams p)
{
    const int32_t b = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (b < p.p.B)
        fork_gather(p, b, lane, 32);
    __syncthreads();
    const bool taken = b < p.p.B && fork_apply(p, b, lane, 32);
    __syncwarp();
    if (taken && lane == 0)
        fork_end(p, b);
}

// ---------------------------------------------------------------------------
// reserve, in one block: whatever it decides depends on all sequences
// ---------------------------------------------------------------------------
constexpr int kReserveThreads = 1024, kReserveWarps = kReserveThreads / 32;
constexpr int kScan = 16;  // pages a thread looks at in a round

// What sequence b asks for: entries [first, mid) are held and will be written to,
// [mid, need) are missing.
struct Wanted {
    int32_t held, first, mid, need;
};

__device__ __forceinline__ Wanted wanted(const ReserveParams& p, int32_t b, bool report,
                                         int32_t len, int32_t n, int32_t held)
{
    const int32_t page = 1 << p.p.page_log2;
    if (len < 0 || len > (int64_t)p.p.max_pages * page || n < 0 || n > p.T || n > len ||
        held < 0 || held > p.p.max_pages) {
        if (report)
            cache_fault(p.p.status, held < 0 || held > p.p.max_pages ? kSiteHeld
                                    : len < 0 || len > (int64_t)p.p.max_pages * page
                                        ? kSiteSeqLen
                                        : kSiteNewLen, b);
        return {0, 0, 0, 0};
    }
    const int32_t need = (len + page - 1) >> p.p.page_log2;
    const int32_t first = n > 0 ? (len - n) >> p.p.page_log2 : need;
    return {held, first, max(first, min(held, need)), max(held, need)};
}

__device__ __forceinline__ int32_t new_rows(const ReserveParams& p, int32_t b)
{
    return p.new_lens ? p.new_lens[b] : p.T;
}

__device__ __forceinline__ Wanted wanted(const ReserveParams& p, int32_t b, bool report)
{
    return wanted(p, b, report, p.p.seq_lens[b], new_rows(p, b), p.p.held[b]);
}

// Calls f(sequence, page, its holders) for the pages that will be written to, a sequence by
// `lanes` threads: four sequences at once, so that their loads (lengths, then entries, then
// holders) are on their way together.  Pages that are none are reported or passed over.
template <class F>
__device__ __forceinline__ void each_written(const ReserveParams& p, int lanes_log2, bool report,
                                             F f)
{
    constexpr int kAtOnce = 4;
    const int32_t lanes = 1 << lanes_log2, mine = threadIdx.x & (lanes - 1);
    const int32_t step = kReserveThreads >> lanes_log2;
    for (int32_t b0 = threadIdx.x >> lanes_log2; b0 < p.p.B; b0 += kAtOnce * step) {
        int32_t len[kAtOnce], n[kAtOnce], held[kAtOnce], id[kAtOnce], refs[kAtOnce];
        Wanted w[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const int32_t b = b0 + k * step;
            len[k] = b < p.p.B ? p.p.seq_lens[b] : 0;
            n[k] = b < p.p.B ? new_rows(p, b) : 0;
            held[k] = b < p.p.B ? p.p.held[b] : 0;
        }
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            w[k] = wanted(p, b0 + k * step, report && mine == 0, len[k], n[k], held[k]);
            w[k].first += mine;
        }
        for (bool more = true; more;) {
            more = false;
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k)
                id[k] = w[k].first < w[k].mid
                            ? p.p.table[(int64_t)(b0 + k * step) * p.p.max_pages + w[k].first]
                            : -1;
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k)
                refs[k] = id[k] >= 0 && id[k] < p.p.npages ? p.p.refs[id[k]] : -1;
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                if (w[k].first < w[k].mid) {
                    if (id[k] >= 0 && id[k] < p.p.npages)
                        f(b0 + k * step, id[k], refs[k]);
                    else if (report)
                        cache_fault(p.p.status, kSitePage, b0 + k * step);
                }
                w[k].first += lanes;
                more |= w[k].first < w[k].mid;
            }
        }
    }
}

// (Pages with one holder have no entries in `writers` and `last`.  A page that is copied has
// two holders or more until its last copy is taken: the copying sequence and one that keeps.)
__device__ __forceinline__ bool is_copied(const ReserveParams& p, int32_t b, int32_t id)
{
    return id >= 0 && id < p.p.npages && p.p.refs[id] > 1 && p.writers[id] > 0 && p.last[id] != b;
}

// Sequence b takes its share of the `total` free pages, by a warp.  (The tests of indexes
// are for lengths that change while the kernel runs.)
__device__ __forceinline__ void take_pages(const ReserveParams& p, int32_t b, int32_t total)
{
    const int lane = threadIdx.x & 31;
    const Wanted w = wanted(p, b, false);
    const int2 at = p.offset[b];
    int32_t* row = p.p.table + (int64_t)b * p.p.max_pages;
    int32_t taken = 0;
    auto take = [&](int32_t i) -> int32_t {
        if (at.x + i >= total)
            return -1;
        const int32_t id = p.free[at.x + i];
        p.p.refs[id] = 1;
        return id;
    };
    for (int32_t e0 = w.first; e0 < w.mid; e0 += 32) {
        const int32_t e = e0 + lane, id = e < w.mid ? row[e] : -1;
        const bool mine = is_copied(p, b, id);
        const uint32_t all = __ballot_sync(0xffffffffu, mine);
        const int32_t i = taken + __popc(all & ((1u << lane) - 1));
        if (mine && at.y + i < p.max_jobs) {
            const int32_t to = take(i);
            row[e] = to;
            p.jobs[at.y + i] = make_int2(id, to);
            atomicSub(p.p.refs + id, 1);
        }
        taken += __popc(all);
    }
    for (int32_t e = w.held + lane; e < w.need; e += 32)
        row[e] = take(taken + e - w.held);
    __syncwarp();
    if (lane == 0 && w.need > w.held)
        p.p.held[b] = w.need;
}

// Exclusive sums of two numbers over the block's threads, and their totals.
__device__ __forceinline__ int2 block_scan(int2 x, int2& total, int2* warp_sums)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int2 y = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, y.x, o), c = __shfl_up_sync(0xffffffffu, y.y, o);
        if (lane >= o)
            y.x += a, y.y += c;
    }
    __syncthreads();  // (the sums of the scan before this one have been read)
    if (lane == 31)
        warp_sums[warp] = y;
    __syncthreads();
    int2 before = make_int2(0, 0);
    total = make_int2(0, 0);
    for (int w = 0; w < kReserveWarps; ++w) {
        const int2 s = warp_sums[w];
        if (w < warp)
            before.x += s.x, before.y += s.y;
        total.x += s.x, total.y += s.y;
    }
    return make_int2(before.x + y.x - x.x, before.y + y.y - x.y);
}

__global__ void __launch_bounds__(kReserveThreads)
    reserve_kernel(const __grid_constant__ ReserveParams p)
{
    __shared__ int2 warp_sums[kReserveWarps];
    __shared__ int32_t counts[kScan * kReserveWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int32_t B = p.p.B;
    // The first round's pages, on their way while it is found out how many are needed.
    int32_t holders[kScan];
    auto look = [&](int64_t base) {
#pragma unroll
        for (int k = 0; k < kScan; ++k) {
            const int64_t id = base + k * kReserveThreads + threadIdx.x;
            holders[k] = id < p.p.npages ? p.p.refs[id] : 1;
        }
    };
    look(0);
    // Pages that will be written to and have other holders: how many of their holders
    // write, and the last of them, which keeps the page if all do.
    bool shared = false;
    each_written(p, p.lanes_log2, true, [&](int32_t, int32_t id, int32_t refs) {
        if (refs > 1) {
            p.last[id] = -1;
            p.writers[id] = 0;
            shared = true;
        }
    });
    shared = __syncthreads_or(shared);
    if (shared) {
        each_written(p, p.lanes_log2, false, [&](int32_t b, int32_t id, int32_t refs) {
            if (refs > 1) {
                atomicMax(p.last + id, b);
                atomicAdd(p.writers + id, 1);
            }
        });
        __syncthreads();
        // (decided once, by the last writer: refs change further down)
        each_written(p, p.lanes_log2, false, [&](int32_t b, int32_t id, int32_t refs) {
            if (refs > 1 && p.last[id] == b && p.writers[id] != refs)
                p.last[id] = INT32_MAX;  // nobody keeps it
        });
        __syncthreads();
    }
    int2 sum = make_int2(0, 0), total;
    const int lanes_log2 = shared ? p.lanes_log2 : 0;  // (else no entry is looked at)
    const int32_t lanes = 1 << lanes_log2, part = threadIdx.x & (lanes - 1);
    for (int32_t b0 = 0; b0 < B; b0 += kReserveThreads >> lanes_log2) {
        const int32_t b = b0 + (threadIdx.x >> lanes_log2);
        int2 mine = make_int2(0, 0);
        if (b < B) {
            const Wanted w = wanted(p, b, false);
            if (shared)
                for (int32_t e = w.first + part; e < w.mid; e += lanes)
                    mine.y += is_copied(p, b, p.p.table[(int64_t)b * p.p.max_pages + e]);
            mine.x = mine.y + (part == 0 ? w.need - w.held : 0);
        }
        const int2 at = block_scan(mine, total, warp_sums);
        if (b < B && part == 0)
            p.offset[b] = make_int2(sum.x + at.x, sum.y + at.y);
        sum.x += total.x;
        sum.y += total.y;
    }
    // The lowest free pages, 32 neighbours a warp at a time.
    int32_t found = 0;
    for (int64_t base = 0; base < p.p.npages && found < sum.x && sum.y <= p.max_jobs;
         base += kScan * kReserveThreads) {
        uint32_t here[kScan];
        if (base > 0)
            look(base);
#pragma unroll
        for (int k = 0; k < kScan; ++k) {
            here[k] = __ballot_sync(0xffffffffu, holders[k] == 0);
            if (lane == 0)
                counts[k * kReserveWarps + warp] = __popc(here[k]);
        }
        __syncthreads();
        const int32_t n = threadIdx.x < kScan * kReserveWarps ? counts[threadIdx.x] : 0;
        const int2 at = block_scan(make_int2(n, 0), total, warp_sums);
        if (threadIdx.x < kScan * kReserveWarps)
            counts[threadIdx.x] = at.x;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kScan; ++k) {
            const int32_t to = found + counts[k * kReserveWarps + warp] +
                               __popc(here[k] & ((1u << lane) - 1));
            if ((here[k] >> lane & 1) && to < sum.x)
                p.free[to] = (int32_t)(base + k * kReserveThreads + threadIdx.x);
        }
        found += total.x;
        __syncthreads();
    }
    const bool refused = found < sum.x || sum.y > p.max_jobs;
    if (threadIdx.x == 0) {
        p.info[0] = refused ? 0 : sum.y;
        p.info[1] = sum.x;
        p.info[2] = refused;
        p.info[3] = 0;
        if (refused)
            cache_fault(p.p.status, kSitePool, sum.x);
    }
    if (refused || !p.here)
        return;
    __syncthreads();  // the list of free pages
    for (int32_t b = warp; b < B; b += kReserveWarps)
        take_pages(p, b, sum.x);
}

// Pages of many sequences, where one block would go through them in many rounds.
__global__ void __launch_bounds__(128) take_kernel(const __grid_constant__ ReserveParams p)
{
    const int32_t b = blockIdx.x * 4 + (threadIdx.x >> 5);
    if (b < p.p.B && !p.info[2])
        take_pages(p, b, p.info[1]);
}

// One warp per sequence.
__global__ void __launch_bounds__(256) trim_kernel(const __grid_constant__ PoolView p)
{
    const int32_t b = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (b >= p.B)
        return;
    const int32_t len = p.seq_lens[b];
    int32_t held;
    if (!pages_held(p, b, held))
        return;
    if (len < 0 || len > (int64_t)p.max_pages << p.page_log2) {
        cache_fault(p.status, kSiteSeqLen, b);
        return;
    }
    const int32_t need = (len + (1 << p.page_log2) - 1) >> p.page_log2;
    for (int32_t e = need + lane; e < held; e += 32)
        release(p, b, p.table[(int64_t)b * p.max_pages + e]);
    __syncwarp();
    if (lane == 0 && need < held)
        p.held[b] = need;
}

// ---------------------------------------------------------------------------
// copies of pages
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) copy_kernel(const __grid_constant__ CopyParams p)
{
    constexpr int kChunk = 1024;  // 16-byte words of a work unit
    const int32_t jobs = min(max(p.info[0], 0), p.max_jobs);
    const int32_t cell = p.c.e4m3 ? 1 : 2;
    const int64_t words = (int64_t)p.c.Hkv * p.c.page * p.c.d * cell / 16;
    const int64_t chunks = (words + kChunk - 1) / kChunk;
    for (int64_t u = blockIdx.x; u < jobs * 2 * chunks; u += gridDim.x) {
        const int64_t job = u / (2 * chunks), rest = u - job * 2 * chunks;
        const bool is_v = rest >= chunks;
        const int64_t w0 = (rest - is_v * chunks) * kChunk;
        const int2 j = p.jobs[job];
        if (j.x < 0 || j.x >= p.c.npages || j.y < 0 || j.y >= p.c.npages) {
            cache_fault(p.c.status, kSitePage, (int)job);
            continue;
        }
        uint8_t* cells = (uint8_t*)(is_v ? p.c.v : p.c.k);
        const uint4* from = (const uint4*)(cells + j.x * p.c.page_stride * cell) + w0;
        uint4* to = (uint4*)(cells + j.y * p.c.page_stride * cell) + w0;
        const int32_t n = (int32_t)min((int64_t)kChunk, words - w0);
        uint4 x[kChunk / 256];
#pragma unroll
        for (int i = 0; i < kChunk / 256; ++i)
            if (i * 256 + (int)threadIdx.x < n)
                x[i] = from[i * 256 + threadIdx.x];
#pragma unroll
        for (int i = 0; i < kChunk / 256; ++i)
            if (i * 256 + (int)threadIdx.x < n)
                to[i * 256 + threadIdx.x] = x[i];
        if (p.c.e4m3 && w0 == 0) {
            float* s = is_v ? p.c.v_scale : p.c.k_scale;
            for (int32_t h = threadIdx.x; h < p.c.Hkv; h += 256)
                s[(int64_t)j.y * p.c.Hkv + h] = s[(int64_t)j.x * p.c.Hkv + h];
        }
    }
}

// ---------------------------------------------------------------------------
// kept rows moved together
// ---------------------------------------------------------------------------
// 16 codes times f
__device__ __forceinline__ uint4 rescaled16(const uint4& w, float f)
{
    const uint32_t in[4] = {w.x, w.y, w.z, w.w};
    uint32_t out[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 a = e4m3x2_float2(in[j] & 0xffffu), c = e4m3x2_float2(in[j] >> 16);
        out[j] = e4m3x4(a.x * f, a.y * f, c.x * f, c.y * f);
    }
    return make_uint4(out[0], out[1], out[2], out[3]);
}

// A block per sequence, head, K or V (and for bf16 cells, which have no scale in common, 64
// bytes of the rows), batch after batch of rows whose places end with a page: row i goes to
// place i and comes from place kept[i] >= i, so that no row of a later batch is overwritten
// before it is read, and no page of one is another's.  Where a batch's rows come from is
// looked up while the batch before is on its way.
//
// Bound by HBM for many rows: half of 16 contexts of up to 8191 rows of 8 heads (269 MB
// moved) 54 us, 4.9 TB/s: single rows are read, every other one.  Batches of twice as many
// rows, half as many blocks on an SM: 69 us; page after page, without looking ahead, 152 us;
// whole rows of bf16, fewer blocks, 81 us, and 32 bytes of them 91 us (before the smaller
// batches).  A path of a few rows takes the chain of loads, 4 us.
constexpr int kCompactThreads = 256, kCompactWords = 8;  // 16-byte words a thread at a time

template <bool F8, int D>
constexpr int kCompactParts = F8 ? 1 : D / 32;
static_assert(kCompactParts<false, 128> == kCompactMaxParts);

template <bool F8, int D>
__global__ void __launch_bounds__(kCompactThreads)
    compact_kernel(const __grid_constant__ CompactParams p)
{
    constexpr int kParts = kCompactParts<F8, D>;
    constexpr int kPerRow = D * (F8 ? 1 : 2) / 16 / kParts;  // 16-byte words of a row
    constexpr int kRows = kCompactThreads * kCompactWords / kPerRow;  // of a batch
    constexpr int kRowWarp = kCompactThreads / kPerRow;  // rows of one word a thread
    __shared__ const uint4* from[2][kRows];              // NULL: no such page
    __shared__ float scale_of[F8 ? 2 : 1][F8 ? kRows : 1];
    __shared__ uint32_t top[F8 ? 2 : 1][F8 ? kRows / 16 + 1 : 1];  // of a batch's pages
    __shared__ int32_t moved_from;
    const uint32_t item = blockIdx.x / kParts;
    const int32_t part = blockIdx.x % kParts;
    const int32_t b = item / (2 * p.c.Hkv);
    const int32_t h = (item - b * 2 * p.c.Hkv) >> 1;
    const bool is_v = item & 1;
    int32_t len, n;
    seq_rows(p.c, p.q_lens, p.T, b, len, n);
    const int32_t a = p.kept_lens ? p.kept_lens[b] : p.A;
    const int32_t* kept = p.kept + (int64_t)b * p.A;
    if (threadIdx.x == 0)
        moved_from = INT32_MAX;
    // All of the list is looked at before the first row moves.
    bool bad = a < 0 || a > p.A || a > n;
    int32_t stays = INT32_MAX;
    if (!bad)
#pragma unroll 4
        for (int32_t i = threadIdx.x; i < a; i += kCompactThreads) {
            const int32_t x = kept[i], before = i > 0 ? kept[i - 1] : -1;
            bad |= x <= before || x >= n;
            if (x != i)
                stays = min(stays, i);
        }
    if (__syncthreads_or(bad)) {
        if (bad)
            cache_fault(p.c.status, kSiteKept, b);
        return;
    }
    if (stays != INT32_MAX)
        atomicMin(&moved_from, stays);
    __syncthreads();
    const int32_t i0 = moved_from, first = len - n;
    if (i0 >= a)
        return;
    const int32_t page = p.c.page, end = first + a;
    uint8_t* cells = (uint8_t*)(is_v ? p.c.v : p.c.k);
    float* scales = is_v ? p.c.v_scale : p.c.k_scale;
    auto row_at = [&](int32_t id, int32_t r) {
        return cells + ((int64_t)id * p.c.page_stride + (((int64_t)h << p.c.page_log2) + r) * D) *
                           (F8 ? 1 : 2) + part * kPerRow * 16;
    };
    auto batch_end = [&](int32_t lo) { return min(end, (lo & ~(page - 1)) + kRows); };
    // Where the rows of [lo, batch_end(lo)) come from, and the largest of their scales for
    // each page that they go to.
    auto look_up = [&](int32_t lo, int set) {
        const int32_t hi = batch_end(lo), start = lo & ~(page - 1);
        for (int32_t r = lo + (int32_t)threadIdx.x; r < hi; r += kCompactThreads) {
            const int32_t j = first + kept[r - first];
            const int32_t id = page_of(p.c, b, j >> p.c.page_log2);
            from[set][r - start] =
                id >= 0 ? reinterpret_cast<const uint4*>(row_at(id, j & (page - 1))) : nullptr;
            if (F8) {
                const float s = id >= 0 ? scales[(int64_t)id * p.c.Hkv + h] : 0.f;
                scale_of[set][r - start] = s;
                atomicMax(&top[set][(r - start) >> p.c.page_log2], __float_as_uint(s));
            }
        }
    };
    auto clear = [&](int set) {
        if (F8)
            for (int i = threadIdx.x; i <= kRows / 16; i += kCompactThreads)
                top[set][i] = 0;
    };
    clear(0);
    __syncthreads();
    look_up(first + i0, 0);
    int set = 0;
    for (int32_t lo = first + i0; lo < end; set ^= 1) {
        const int32_t hi = batch_end(lo), start = lo & ~(page - 1);
        __syncthreads();  // the rows are looked up; the other set has been used
        if (F8) {
            clear(set ^ 1);
            __syncthreads();
        }
        const int32_t at = threadIdx.x / kPerRow, word = threadIdx.x % kPerRow;
        uint4 x[kCompactWords];
#pragma unroll
        for (int k = 0; k < kCompactWords; ++k) {
            const int32_t r = start + at + k * kRowWarp;
            if (r >= lo && r < hi && from[set][r - start])
                x[k] = from[set][r - start][word];
        }
        if (hi < end)
            look_up(hi, set ^ 1);
        // The rows of the first page that stay: to the page's new scale.
        const int32_t to0 = page_of(p.c, b, lo >> p.c.page_log2);
        float old = 0.f;
        if (F8 && lo > start && to0 >= 0)
            old = scales[(int64_t)to0 * p.c.Hkv + h];
        __syncthreads();  // all rows of the batch have been read, and the old scale
        if (F8 && lo > start && to0 >= 0) {
            const float s = fmaxf(old, __uint_as_float(top[set][0]));
            if (s != old) {
                const float f = old / s;
                for (int32_t w = threadIdx.x; w < (lo - start) * kPerRow; w += kCompactThreads) {
                    uint4* cell = reinterpret_cast<uint4*>(row_at(to0, w / kPerRow)) + w % kPerRow;
                    *cell = rescaled16(*cell, f);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < kCompactWords; ++k) {
            const int32_t r = start + at + k * kRowWarp;
            if (r < lo || r >= hi || !from[set][r - start])
                continue;
            const int32_t pg = r >> p.c.page_log2, id = page_of(p.c, b, pg);
            if (id < 0)
                continue;
            if (F8) {
                float s = __uint_as_float(top[set][(r - start) >> p.c.page_log2]);
                if (pg << p.c.page_log2 == start)
                    s = fmaxf(s, old);
                const float mine = scale_of[set][r - start];
                if (mine != s)
                    x[k] = rescaled16(x[k], mine / s);
                // (the page's first row here, or its first one at all)
                if (word == 0 && (r == lo || (r & (page - 1)) == 0))
                    scales[(int64_t)id * p.c.Hkv + h] = s;
            }
            reinterpret_cast<uint4*>(row_at(id, r & (page - 1)))[word] = x[k];
        }
        lo = hi;
    }
}

}  // namespace

cudaError_t launch_pages_fork(const ForkParams& p, cudaStream_t stream)
{
    if (p.p.B <= kForkHere && p.p.max_pages <= 1024) {  // (32 rounds of a warp)
        fork_kernel<<<1, 32 * kForkHere, 0, stream>>>(p);
        return cudaGetLastError();
    }
    const unsigned parts = max(1, min(8, p.p.max_pages / 2048));
    fork_gather_kernel<<<dim3(p.p.B, parts), 256, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    fork_apply_kernel<<<p.p.B, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_pages_reserve(ReserveParams& p, cudaStream_t stream)
{
    // One warp a sequence, in two rounds at most; where there are more, in blocks of their
    // own behind this one.
    p.here = p.p.B <= 2 * kReserveWarps;
    // A thread for each page that T rows can reach, a warp at most.
    const int32_t pages = p.T > 0 ? ((p.T - 1) >> p.p.page_log2) + 2 : 1;
    for (p.lanes_log2 = 0; p.lanes_log2 < 5 && 1 << p.lanes_log2 < pages;)
        ++p.lanes_log2;
    reserve_kernel<<<1, kReserveThreads, 0, stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || p.here)
        return e;
    take_kernel<<<(p.p.B + 3) / 4, 128, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_pages_trim(const PoolView& p, cudaStream_t stream)
{
    trim_kernel<<<(p.B + 7) / 8, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_cache_copy(const CopyParams& p, int num_sms, cudaStream_t stream)
{
    const int64_t words = (int64_t)p.c.Hkv * p.c.page * p.c.d * (p.c.e4m3 ? 1 : 2) / 16;
    const int64_t units = p.max_jobs * 2 * ((words + 1023) / 1024);
    copy_kernel<<<(unsigned)min(units, (int64_t)num_sms * 8), 256, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_cache_compact(const CompactParams& p, cudaStream_t stream)
{
    const unsigned heads = 2u * p.c.Hkv * p.c.B;
    if (p.c.e4m3)
        p.c.d == 128 ? compact_kernel<true, 128><<<heads, kCompactThreads, 0, stream>>>(p)
                     : compact_kernel<true, 64><<<heads, kCompactThreads, 0, stream>>>(p);
    else if (p.c.d == 128)
        compact_kernel<false, 128>
            <<<heads * kCompactParts<false, 128>, kCompactThreads, 0, stream>>>(p);
    else
        compact_kernel<false, 64>
            <<<heads * kCompactParts<false, 64>, kCompactThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace dfa
