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

__device__ __forceinline__ void release(const PoolView& p, int32_t b, int32_t id)
{
    if (pool_page(p, b, id) && atomicSub(p.refs + id, 1) <= 0)
        cache_fault(p.status, kSiteRefs, b);
}

// ---------------------------------------------------------------------------
// fork: what the sequences will hold, gathered before anything changes; then taken over
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) fork_gather_kernel(const __grid_constant__ ForkParams p)
{
    const int32_t b = blockIdx.x, src = p.src[b];
    if (src == b)
        return;
    int32_t held = 0, len = 0;
    bool ok = src >= -1 && src < p.p.B;
    if (!ok)
        cache_fault(p.p.status, kSiteSource, b);
    else if (src >= 0) {
        ok = pages_held(p.p, src, held);
        len = p.p.seq_lens[src];
    }
    if (threadIdx.x == 0 && blockIdx.y == 0) {
        p.held[b] = ok ? held : -1;  // -1: stays as it is
        p.lens[b] = len;
    }
    if (!ok)
        return;
    const int32_t* from = p.p.table + (int64_t)src * p.p.max_pages;
    int32_t* to = p.rows + (int64_t)b * p.p.max_pages;
    for (int32_t e = blockIdx.y * blockDim.x + threadIdx.x; e < held; e += gridDim.y * blockDim.x)
        to[e] = from[e];
}

// (Entries that stay, the shared beginning of beams for one, cost no atomics.)
__global__ void __launch_bounds__(256) fork_apply_kernel(const __grid_constant__ ForkParams p)
{
    const int32_t b = blockIdx.x;
    if (p.src[b] == b)
        return;
    const int32_t held = p.held[b];
    int32_t old_held;
    if (held < 0 || !pages_held(p.p, b, old_held))
        return;
    int32_t* row = p.p.table + (int64_t)b * p.p.max_pages;
    const int32_t* from = p.rows + (int64_t)b * p.p.max_pages;
    const int32_t end = max(held, old_held);
    for (int32_t e = threadIdx.x; e < end; e += blockDim.x) {
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
    __syncthreads();  // everyone has read what it held
    if (threadIdx.x == 0) {
        p.p.held[b] = held;
        p.p.seq_lens[b] = p.lens[b];
    }
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

__device__ __forceinline__ Wanted wanted(const ReserveParams& p, int32_t b, bool report)
{
    const int32_t len = p.p.seq_lens[b], n = p.new_lens ? p.new_lens[b] : p.T;
    const int32_t held = p.p.held[b];
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
    auto entry = [&](int32_t b, int32_t e) { return p.p.table[(int64_t)b * p.p.max_pages + e]; };
    // Pages that will be written to and have other holders: how many of their holders
    // write, and the last of them, which keeps the page if all do.
    for (int32_t b = threadIdx.x; b < B; b += kReserveThreads) {
        const Wanted w = wanted(p, b, true);
        for (int32_t e = w.first; e < w.mid; ++e) {
            const int32_t id = entry(b, e);
            if (pool_page(p.p, b, id)) {
                p.last[id] = -1;
                p.writers[id] = 0;
            }
        }
    }
    __syncthreads();
    for (int32_t b = threadIdx.x; b < B; b += kReserveThreads) {
        const Wanted w = wanted(p, b, false);
        for (int32_t e = w.first; e < w.mid; ++e) {
            const int32_t id = entry(b, e);
            if (id >= 0 && id < p.p.npages && p.p.refs[id] > 1) {
                atomicMax(p.last + id, b);
                atomicAdd(p.writers + id, 1);
            }
        }
    }
    __syncthreads();
    // (decided once, by the last writer: refs change further down)
    for (int32_t b = threadIdx.x; b < B; b += kReserveThreads) {
        const Wanted w = wanted(p, b, false);
        for (int32_t e = w.first; e < w.mid; ++e) {
            const int32_t id = entry(b, e);
            if (id >= 0 && id < p.p.npages && p.last[id] == b && p.writers[id] != p.p.refs[id])
                p.last[id] = INT32_MAX;  // nobody keeps it
        }
    }
    __syncthreads();
    auto copied = [&](int32_t b, int32_t id) {
        return id >= 0 && id < p.p.npages && p.writers[id] > 0 && p.last[id] != b;
    };
    int2 sum = make_int2(0, 0), total;
    for (int32_t b0 = 0; b0 < B; b0 += kReserveThreads) {
        const int32_t b = b0 + threadIdx.x;
        int2 mine = make_int2(0, 0);
        if (b < B) {
            const Wanted w = wanted(p, b, false);
            for (int32_t e = w.first; e < w.mid; ++e)
                mine.y += copied(b, entry(b, e));
            mine.x = mine.y + w.need - w.held;
        }
        const int2 at = block_scan(mine, total, warp_sums);
        if (b < B)
            p.offset[b] = make_int2(sum.x + at.x, sum.y + at.y);
        sum.x += total.x;
        sum.y += total.y;
    }
    // The lowest free pages, 32 neighbours a warp at a time.
    int32_t found = 0;
    for (int64_t base = 0; base < p.p.npages && found < sum.x && sum.y <= p.max_jobs;
         base += kScan * kReserveThreads) {
        uint32_t here[kScan];
#pragma unroll
        for (int k = 0; k < kScan; ++k) {
            const int64_t id = base + k * kReserveThreads + threadIdx.x;
            here[k] = id < p.p.npages ? (uint32_t)p.p.refs[id] : 1u;
        }
#pragma unroll
        for (int k = 0; k < kScan; ++k) {
            here[k] = __ballot_sync(0xffffffffu, here[k] == 0);
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
    if (refused)
        return;
    __syncthreads();  // the list of free pages
    for (int32_t b = warp; b < B; b += kReserveWarps) {
        const Wanted w = wanted(p, b, false);
        const int2 at = p.offset[b];
        int32_t* row = p.p.table + (int64_t)b * p.p.max_pages;
        int32_t taken = 0;
        // (the tests of indexes are for lengths that change while the kernel runs)
        auto take = [&](int32_t i) -> int32_t {
            if (at.x + i >= sum.x)
                return -1;
            const int32_t id = p.free[at.x + i];
            p.p.refs[id] = 1;
            return id;
        };
        for (int32_t e0 = w.first; e0 < w.mid; e0 += 32) {
            const int32_t e = e0 + lane, id = e < w.mid ? row[e] : -1;
            const bool mine = copied(b, id);
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
    if (len < 0) {
        cache_fault(p.status, kSiteSeqLen, b);
        return;
    }
    const int32_t need = (int32_t)(((int64_t)len + (1 << p.page_log2) - 1) >> p.page_log2);
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

// A block per sequence, head and K or V, page after page of where the rows go to: row
// i goes to place i and comes from place kept[i] >= i, so that no row of a later page
// is overwritten before it is read.
template <bool F8, int D>
__global__ void __launch_bounds__(256) compact_kernel(const __grid_constant__ CompactParams p)
{
    constexpr int kPerRow = D * (F8 ? 1 : 2) / 16;       // 16-byte words of a row
    constexpr int kMost = (128 * kPerRow + 255) / 256;   // of a page, a thread
    __shared__ int32_t moved_from;
    __shared__ uint32_t top;
    const int32_t b = blockIdx.x / (2 * p.c.Hkv);
    const int32_t h = (blockIdx.x - b * 2 * p.c.Hkv) >> 1;
    const bool is_v = blockIdx.x & 1;
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
        for (int32_t i = threadIdx.x; i < a; i += 256) {
            const int32_t x = kept[i];
            bad |= x < 0 || x >= n || (i > 0 && kept[i - 1] >= x);
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
                           (F8 ? 1 : 2);
    };
    for (int32_t pg = (first + i0) >> p.c.page_log2; pg << p.c.page_log2 < end; ++pg) {
        const int32_t start = pg << p.c.page_log2;
        const int32_t lo = max(first + i0, start), hi = min(end, start + page);
        const int32_t to = page_of(p.c, b, pg);
        uint4 x[kMost];
        float s[kMost];
        bool there[kMost];
        float mine = 0.f;
#pragma unroll
        for (int k = 0; k < kMost; ++k) {
            const int32_t w = k * 256 + threadIdx.x, r = lo + w / kPerRow;
            there[k] = false;
            if (r >= hi)
                continue;
            const int32_t from = first + kept[r - first];
            const int32_t id = page_of(p.c, b, from >> p.c.page_log2);
            there[k] = id >= 0 && to >= 0;
            if (!there[k])
                continue;
            x[k] = reinterpret_cast<const uint4*>(row_at(id, from & (page - 1)))[w % kPerRow];
            if (F8) {
                s[k] = scales[(int64_t)id * p.c.Hkv + h];
                mine = fmaxf(mine, s[k]);
            }
        }
        float scale = 1.f;
        if (F8) {
            const float old = to >= 0 ? scales[(int64_t)to * p.c.Hkv + h] : 1.f;
            if (threadIdx.x == 0)
                top = 0;
            __syncthreads();
            atomicMax(&top, __float_as_uint(lo > start ? fmaxf(mine, old) : mine));
            __syncthreads();
            scale = __uint_as_float(top);
            if (to >= 0 && lo > start && scale != old) {
                // the rows that stay, to the new scale
                const float f = old / scale;
                for (int32_t w = threadIdx.x; w < (lo - start) * kPerRow; w += 256) {
                    uint4* cell = reinterpret_cast<uint4*>(row_at(to, w / kPerRow)) + w % kPerRow;
                    *cell = rescaled16(*cell, f);
                }
            }
            if (threadIdx.x == 0 && to >= 0 && scale > 0.f)
                scales[(int64_t)to * p.c.Hkv + h] = scale;
        }
        __syncthreads();  // all rows of the page have been read, and the old scale
#pragma unroll
        for (int k = 0; k < kMost; ++k) {
            const int32_t w = k * 256 + threadIdx.x, r = lo + w / kPerRow;
            if (!there[k])
                continue;
            if (F8 && s[k] != scale)
                x[k] = rescaled16(x[k], s[k] / scale);
            reinterpret_cast<uint4*>(row_at(to, r - start))[w % kPerRow] = x[k];
        }
        __syncthreads();
    }
}

}  // namespace

cudaError_t launch_pages_fork(const ForkParams& p, cudaStream_t stream)
{
    const unsigned parts = max(1, min(8, p.p.max_pages / 2048));
    fork_gather_kernel<<<dim3(p.p.B, parts), 256, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    fork_apply_kernel<<<p.p.B, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_pages_reserve(const ReserveParams& p, cudaStream_t stream)
{
    reserve_kernel<<<1, kReserveThreads, 0, stream>>>(p);
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
    const unsigned grid = 2u * p.c.Hkv * p.c.B;
    if (p.c.e4m3)
        p.c.d == 128 ? compact_kernel<true, 128><<<grid, 256, 0, stream>>>(p)
                     : compact_kernel<true, 64><<<grid, 256, 0, stream>>>(p);
    else
        p.c.d == 128 ? compact_kernel<false, 128><<<grid, 256, 0, stream>>>(p)
                     : compact_kernel<false, 64><<<grid, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace dfa
