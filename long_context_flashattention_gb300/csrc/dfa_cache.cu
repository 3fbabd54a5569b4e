// dfa_cache.cu -- the paged key/value cache: append of new rows (keys rotated,
// both quantised to 8 bits with a power-of-two scale per page and head, or kept
// in bf16) together with the rotation of the queries that go with them, and
// gather of cached rows into contiguous bf16.
//
// Both are HBM-bound for long inputs (a few operations per feature) and bound
// by the chain of dependent loads (length -> page -> scale -> rows) for one
// token.  Two kinds of work, in one launch:
//
// Page jobs (8-bit cells).  A page's scale needs the largest value of all its
// new rows before the first is stored, so a group of threads takes the rows of one
// page and head, a 16-feature unit of a row each, and holds them in registers
// in between: every row is read once.  The group keeps its rows' cos and sin and
// goes through several heads with them, the next two heads' rows on their way into
// shared memory (one head ahead in registers, which then spill: 143 and 302 us for the
// 32K prompts below; three, four and six heads: 133, 137, 164 where two took 132).
//
// Measured: a 32K bf16 prompt of 3 x 32 heads of 128, 239 us, 6.7 TB/s; into 8 bits
// with 8 key/value heads 128 us, 5.7 TB/s, with 32 248 us, 5.4 TB/s (a group waits for
// its largest value between loads and stores); ragged chunks of 0..1000 tokens into
// 16-row pages, 28 MB, 11.1 us (the launch and the chain of loads, and between them
// instruction issue 60 % of the time, warps of a page at its barrier for the rest); one
// token of 64 sequences 4.1 us.
// Gather of two sequences of up to 64K rows of 8 heads, 604 MB: 81.5 us (part of what it
// writes is still in L2 when it ends).
//
// Row items (queries; K and V too in a bf16 cache, where rows are independent).
// A warp takes one token and several heads; its lanes compute the token's
// cos and sin once between them.
#include "dfa_serve.cuh"

namespace dfa {

namespace {

constexpr int kBatch = 2;     // rows of an item in flight per lane
constexpr int kSlots = 64;    // shared memory of a thread of a page job: two heads' units

// 16 bytes into the thread's own slot of shared memory
__device__ __forceinline__ void copy16(uint32_t to, const void* from)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}

__device__ __forceinline__ uint4 load16(uint32_t at)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
}

// codes of x / s; a NaN stays one
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float inv)
{
    return make_uint2(e4m3x4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv),
                      e4m3x4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv));
}

// The largest value that a cell may stand for: from scale 2^120 on, bf16's largest values
// would be rounded up to 2^128, an infinity.
constexpr float kLargest = 240.f * 0x1p120f;

// Infinities become NaN (the conversion would store them as the largest finite
// cell), and what is beyond the largest value that value.
__device__ __forceinline__ void bound_values(float (&x)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (fabsf(x[i]) > kLargest)
            x[i] = fabsf(x[i]) == INFINITY ? NAN : copysignf(kLargest, x[i]);
}

// Largest |x|, NaN left out (fmaxf does)
__device__ __forceinline__ float abs_max8(float m, const float (&x)[8])
{
#pragma unroll
    for (int i = 0; i < 8; i += 2)
        m = fmaxf(m, fmaxf(fabsf(x[i]), fabsf(x[i + 1])));
    return m;
}

// Row items of a block.  Rows of a token: Hq queries, then (bf16 cache) Hkv keys
// and Hkv values.
template <bool F8, int D>
__device__ __forceinline__ void row_items(const AppendParams& p, const uint64_t* turns,
                                          uint32_t item, uint32_t stride)
{
    constexpr int UNITS = D / 16, kStep = 32 / UNITS;
    const int lane = threadIdx.x & 31;
    const int u = lane & (UNITS - 1), h_lane = lane / UNITS;
    const int32_t Hk = F8 ? 0 : p.c.Hkv, rows = p.Hq + 2 * Hk;
    const uint32_t per_token = (rows + p.item_heads - 1) / p.item_heads;
    int f0, f1;
    const bool turned = unit_runs<8>(p.t, D, u, f0, f1);
    const SharedAngles<8, UNITS, kStep> angles(p.t, turns);
    for (; item < p.items; item += stride) {
        const uint32_t token = item / per_token;
        const int32_t h0 = (int32_t)(item - token * per_token) * p.item_heads;
        const int32_t h1 = min(h0 + p.item_heads, rows);
        const int32_t b = token / (uint32_t)p.T, t = token - (uint32_t)b * (uint32_t)p.T;
        int32_t len, n;
        seq_rows(p.c, p.new_lens, p.T, b, len, n);
        if (t >= n)
            continue;
        const int32_t pos = len - n + t;
        const int32_t turn = p.positions ? p.positions[token] : pos;  // (token: b * T + t)
        const bool stores = !F8 && h1 > p.Hq;
        int32_t id = stores ? page_entry(p.c, b, pos >> p.c.page_log2) : 0;
        float cs[8], sn[8];
        for (int32_t h = h0; h < h1; h += kBatch * kStep) {
            Run<__nv_bfloat16> r[kBatch][2];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int32_t hk = h + h_lane + k * kStep;
                if (hk >= h1)
                    continue;
                const bool is_v = hk >= p.Hq + Hk;
                const Rows& src = F8 || hk < p.Hq ? p.q : is_v ? p.v : p.k;
                const int32_t hs = F8 || hk < p.Hq ? hk : hk - p.Hq - (is_v ? Hk : 0);
                const __nv_bfloat16* from =
                    (const __nv_bfloat16*)src.p + b * src.sb + hs * src.sh + t * src.sl;
                r[k][0].load(from + f0);
                r[k][1].load(from + f1);
            }
            if (h == h0) {  // while the first rows are on their way
                if (p.t.half && h0 < p.Hq + Hk)  // (not for values alone)
                    angles.at(turn, 1.f, cs, sn);
                if (stores && !is_page(p.c, b, id))
                    id = -1;
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int32_t hk = h + h_lane + k * kStep;
                if (hk >= h1)
                    continue;
                if (turned && hk < p.Hq + Hk) {
                    float a[8], c[8];
                    r[k][0].get(a);
                    r[k][1].get(c);
                    unit_rotate<8>(p.t, cs, sn, a, c);
                    r[k][0].set(a);
                    r[k][1].set(c);
                }
                __nv_bfloat16* to;
                if (F8 || hk < p.Hq) {
                    to = (__nv_bfloat16*)p.q_out.p + b * p.q_out.sb + hk * p.q_out.sh +
                         t * p.q_out.sl;
                } else {
                    if (id < 0)
                        continue;
                    const bool is_v = hk >= p.Hq + Hk;
                    const int32_t hc = hk - p.Hq - (is_v ? Hk : 0);
                    to = (__nv_bfloat16*)(is_v ? p.c.v : p.c.k) + (int64_t)id * p.c.page_stride +
                         (((int64_t)hc << p.c.page_log2) + (pos & (p.c.page - 1))) * D;
                }
                r[k][0].store(to + f0);
                r[k][1].store(to + f1);
            }
        }
    }
}

// Barrier of one group of threads of the block (barrier 0 is the block's).
__device__ __forceinline__ void group_sync(int group, int threads)
{
    if (threads <= 32)
        __syncwarp();
    else
        asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(threads) : "memory");
}

// Largest value of the group; `set` alternates between two sets of smem words,
// so that one barrier is enough.
__device__ __forceinline__ float group_max(float m, int group, int thread, int threads,
                                           uint32_t (*words)[32], int& set)
{
    // (the bits of floats that are not negative are ordered as they are)
    uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
    if (threads > 32) {
        set ^= 16;
        uint32_t* w = words[set + group];
        if ((thread & 31) == 0)
            w[thread >> 5] = bits;
        group_sync(group, threads);
        const int lane = thread & 31;
        bits = __reduce_max_sync(0xffffffffu, lane < threads / 32 ? w[lane] : 0u);
    }
    return __uint_as_float(bits);
}

// One page job: K or V rows of one page, job_heads heads.  Every thread of the
// group takes the same way through it.
template <int D>
__device__ __forceinline__ void page_job(const AppendParams& p, uint32_t job, int group,
                                         int thread, const uint64_t* turns, uint32_t (*words)[32],
                                         int& set, uint32_t slots)
{
    constexpr int UNITS = D / 16;
    const uint32_t head_jobs = (p.c.Hkv + p.job_heads - 1) / p.job_heads;
    const uint32_t per_seq = 2 * head_jobs * p.pages;
    const int32_t b = job / per_seq;
    uint32_t i = job - b * per_seq;
    const int32_t ip = i % (uint32_t)p.pages;
    i /= (uint32_t)p.pages;
    const int32_t is_v = i >= head_jobs;
    const int32_t h0 = (i - is_v * head_jobs) * p.job_heads;
    // One look at the lengths for the whole group, whose barriers everyone has to
    // reach.
    const int threads = p.job_threads;
    int32_t len, n;
    if (thread < 32)
        seq_rows(p.c, p.new_lens, p.T, b, len, n);
    if (threads > 32) {
        set ^= 16;
        uint32_t* w = words[set + group];
        if (thread == 0) {
            w[0] = len;
            w[1] = n;
        }
        group_sync(group, threads);
        len = w[0];
        n = w[1];
    }
    const int32_t first = len - n;                          // first new row
    const int32_t pg = (first >> p.c.page_log2) + ip;       // page of the sequence
    const int32_t start = pg << p.c.page_log2;
    const int32_t lo = max(first, start);                   // rows [lo, hi) are new
    const int32_t hi = min(len, start + p.c.page);
    if (lo >= hi)
        return;
    int32_t id = page_entry(p.c, b, pg);
    const Rows& src = is_v ? p.v : p.k;
    const int32_t there = lo - start;        // rows of the page stored before
    const int32_t u = thread & (UNITS - 1);  // threads is a multiple of UNITS
    const int32_t row = lo + thread / UNITS;
    const bool mine = row < hi;
    int f0, f1;
    const bool turned = unit_runs<8>(p.t, D, u, f0, f1) && !is_v;
    float cs[8], sn[8];
    const __nv_bfloat16* x = (const __nv_bfloat16*)src.p + b * src.sb + h0 * src.sh +
                             (row - first) * src.sl + f0;
    const int32_t run1 = f1 - f0;                  // from the first run to the second
    const int32_t at0 = (row - start) * D + f0;    // the first run's cells
    const int32_t h1 = min(h0 + p.job_heads, p.c.Hkv);
    // rows of the next heads, in slots of the thread's own
    const uint32_t half = blockDim.x * 16;
    uint32_t slot = slots + threadIdx.x * 16;
    int32_t step = 2 * half;  // to the other slot
    auto fetch = [&](uint32_t at, bool there) {
        if (mine && there) {
            copy16(at, x);
            copy16(at + half, x + run1);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        x += src.sh;
    };
    fetch(slot, true);
    fetch(slot + step, h0 + 1 < h1);
    const bool stores = is_page(p.c, b, id);  // if not, on to the barriers all the same
    if (!stores)
        id = 0;
    float* scales = (is_v ? p.c.v_scale : p.c.k_scale) + (int64_t)id * p.c.Hkv;
    uint8_t* cells = (uint8_t*)(is_v ? p.c.v : p.c.k) + (int64_t)id * p.c.page_stride +
                     ((int64_t)h0 << p.c.page_log2) * D;
    for (int32_t h = h0; h < h1; ++h, cells += p.c.page * D) {
        const float old = there > 0 && stores ? scales[h] : 0.f;
        if (h == h0 && turned && mine) {
            const int32_t turn =
                p.positions ? p.positions[(int64_t)b * p.T + row - first] : row;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                pair_angle(turns[unit_pair<8>(p.t, u, j)], p.t.gain, turn, 1.f, cs[j], sn[j]);
        }
        float a[8], c[8], amax = 0.f;
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        if (mine) {
            Run<__nv_bfloat16> r0, r1;
            r0.w = load16(slot);
            r1.w = load16(slot + half);
            r0.get(a);
            r1.get(c);
            if (turned)
                unit_rotate<8>(p.t, cs, sn, a, c);
            amax = abs_max8(abs_max8(0.f, a), c);
        }
        fetch(slot, h + 2 < h1);
        slot += step;
        step = -step;
        amax = group_max(amax, group, thread, threads, words, set);
        if (amax > kLargest) {  // (rare) once more, over bounded values
            if (mine) {
                bound_values(a);
                bound_values(c);
            }
            amax = group_max(mine ? abs_max8(abs_max8(0.f, a), c) : 0.f, group, thread, threads,
                             words, set);
        }
        const float s = fmaxf(old, pow2_scale(amax));
        const float inv = 1.f / s;  // exact: a power of two (or a scale of the caller's)
        if (s != old && stores) {
            if (there > 0) {
                // raise the rows that are there to the new scale: exact but for
                // cells that become subnormal
                const float f = old * inv;
                for (int32_t v = thread; v < there * D / 16; v += threads) {
                    uint4* cell = reinterpret_cast<uint4*>(cells) + v;
                    const uint4 w = *cell;
                    const uint32_t in[4] = {w.x, w.y, w.z, w.w};
                    uint32_t out[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 q0 = e4m3x2_float2(in[j] & 0xffffu);
                        const float2 q1 = e4m3x2_float2(in[j] >> 16);
                        out[j] = e4m3x4(q0.x * f, q0.y * f, q1.x * f, q1.y * f);
                    }
                    *cell = make_uint4(out[0], out[1], out[2], out[3]);
                }
            }
            // everyone has read the old scale (the barrier, or the warp's shuffles)
            if (threads <= 32)
                __syncwarp();
            if (thread == 0)
                scales[h] = s;
        }
        if (mine && stores) {
            *reinterpret_cast<uint2*>(cells + at0) = codes8(a, inv);
            *reinterpret_cast<uint2*>(cells + at0 + run1) = codes8(c, inv);
        }
    }
}

template <bool F8, int D>
__global__ void __launch_bounds__(F8 ? 1024 : 256, F8 ? 1 : 3)
    cache_append_kernel(const __grid_constant__ AppendParams p)
{
    __shared__ uint64_t turns[64];  // lanes read different entries: not from the parameters
    // A decode of few blocks behind this kernel may be launched already, and waits (the
    // two, one sequence of 1000 rows, in a graph: 12.7 -> 12.3 us).
    cudaTriggerProgrammaticLaunchCompletion();
    if (threadIdx.x < 64)
        turns[threadIdx.x] = p.t.turn[threadIdx.x];
    __syncthreads();
    if (F8 && (int32_t)blockIdx.x < p.job_blocks) {
        __shared__ uint32_t words[32][32];
        extern __shared__ uint4 slots[];
        const int groups = blockDim.x / p.job_threads;
        const int group = threadIdx.x / p.job_threads;
        int set = 0;
        for (uint32_t job = blockIdx.x * groups + group; job < p.jobs;
             job += p.job_blocks * groups)
            page_job<D>(p, job, group, threadIdx.x - group * p.job_threads, turns, words, set,
                        smem_u32(slots));
        return;
    }
    const int warps = blockDim.x >> 5;
    row_items<F8, D>(p, turns, (blockIdx.x - p.job_blocks) * warps + (threadIdx.x >> 5),
                     (gridDim.x - p.job_blocks) * warps);
}

// One block per (page of the range, head, sequence); K and V.
template <typename CELL>
__global__ void __launch_bounds__(128) cache_gather_kernel(const __grid_constant__ GatherParams p)
{
    constexpr bool k8 = sizeof(CELL) == 1;
    int64_t i = blockIdx.x;
    const int32_t pg = p.page0 + (int32_t)(i % p.pages);
    i /= p.pages;
    const int32_t h = (int32_t)(i % p.c.Hkv), b = (int32_t)(i / p.c.Hkv);
    int32_t len, n;
    seq_rows(p.c, nullptr, 0, b, len, n);
    const int64_t start = (int64_t)pg * p.c.page;
    const int64_t lo = max(p.pos0, start);
    const int64_t hi = min(min((int64_t)len, p.pos0 + p.L), start + p.c.page);
    if (lo >= hi)
        return;
    const int32_t id = page_of(p.c, b, pg);
    if (id < 0)
        return;
    const int32_t d = p.c.d;
    const int32_t vecs = (int32_t)(hi - lo) * d / 8;  // 8 features each
    const int64_t from = (int64_t)id * p.c.page_stride + ((int64_t)h * p.c.page + lo - start) * d;
    const int64_t to = (((int64_t)b * p.c.Hkv + h) * p.L + lo - p.pos0) * d;
#pragma unroll
    for (int is_v = 0; is_v < 2; ++is_v) {
        __nv_bfloat16* out = (__nv_bfloat16*)(is_v ? p.v_out : p.k_out);
        if (!out)
            continue;
        const CELL* cells = (const CELL*)(is_v ? p.c.v : p.c.k) + from;
        const float s =
            k8 ? __ldg((is_v ? p.c.v_scale : p.c.k_scale) + (int64_t)id * p.c.Hkv + h) : 1.f;
        for (int32_t v = threadIdx.x; v < vecs; v += blockDim.x) {
            if (k8) {
                const uint2 w = __ldg(reinterpret_cast<const uint2*>(cells) + v);
                const float2 q0 = e4m3x2_float2(w.x & 0xffffu), q1 = e4m3x2_float2(w.x >> 16);
                const float2 q2 = e4m3x2_float2(w.y & 0xffffu), q3 = e4m3x2_float2(w.y >> 16);
                reinterpret_cast<uint4*>(out + to)[v] =
                    make_uint4(pack_bf16x2(q0.x * s, q0.y * s), pack_bf16x2(q1.x * s, q1.y * s),
                               pack_bf16x2(q2.x * s, q2.y * s), pack_bf16x2(q3.x * s, q3.y * s));
            } else {
                reinterpret_cast<uint4*>(out + to)[v] =
                    __ldg(reinterpret_cast<const uint4*>(cells) + v);
            }
        }
    }
}

}  // namespace

// Work per job, item and block.  Angles are computed once per job or item, so
// each takes as many heads as leave enough threads to fill the SMs; blocks take
// several, a grid's worth at a time.  Measured (8-bit, 32 and 8 heads; jobs for 1024
// threads and items for 64 warps an SM, 512 and 32, 384 and 24, 256 and 8; us): 1024
// tokens 10.3, 10.3, 7.6, 7.8, 2048 17.3, 12.3, 10.3, 10.3, 4096 23.3, 18.6, 18.0;
// ragged chunks of 0..1000 tokens of 16 sequences (d 64) 13.1, 11.1, 11.1, 11.5.
// bf16, items for 24 and 12 warps: 512 tokens 6.1, 4.9, 2048 11.1, 8.6.  Item blocks
// for 4096 threads an SM (a 32K bf16 prompt of 32 heads) 242 us, 2048 249; job blocks
// for 1024 and 2048: 128.7, 129.4.
cudaError_t launch_cache_append(AppendParams& p, int num_sms, cudaStream_t stream)
{
    const int units = p.c.d / 16, step = 32 / units;
    const int64_t tokens = (int64_t)p.c.B * p.T;
    int threads = 256;
    if (p.c.e4m3) {
        const int rows = min(p.T, p.c.page);
        p.job_threads = 32;
        while (p.job_threads < rows * units)
            p.job_threads *= 2;
        threads = max(threads, p.job_threads);
        const int64_t pages = (int64_t)p.c.B * 2 * p.pages;  // of one head
        p.job_heads = 8;
        while (p.job_heads > 1 &&
               pages * ((p.c.Hkv + p.job_heads - 1) / p.job_heads) * p.job_threads <
                   (int64_t)num_sms * 384)
            p.job_heads /= 2;
        p.jobs = (uint32_t)(pages * ((p.c.Hkv + p.job_heads - 1) / p.job_heads));
        const int groups = threads / p.job_threads;
        p.job_blocks = (int32_t)min((p.jobs + groups - 1) / groups, num_sms * 1024u / threads);
    }
    const int rows = p.Hq + (p.c.e4m3 ? 0 : 2 * p.c.Hkv);
    int64_t item_blocks = 0;
    if (rows > 0) {
        p.item_heads = 16 * kBatch * step;
        while (p.item_heads > step &&
               tokens * ((rows + p.item_heads - 1) / p.item_heads) < (int64_t)num_sms * (p.c.e4m3 ? 24 : 12))
            p.item_heads /= 2;
        p.items = (uint32_t)(tokens * ((rows + p.item_heads - 1) / p.item_heads));
        item_blocks = min((p.items + threads / 32 - 1) / (threads / 32),
                          num_sms * (p.c.e4m3 ? 2048u : 4096u) / threads);
    }
    const unsigned blocks = (unsigned)(p.job_blocks + item_blocks);
    if (!p.c.e4m3) {
        auto* kernel = units == 8 ? cache_append_kernel<false, 128> : cache_append_kernel<false, 64>;
        kernel<<<blocks, threads, 0, stream>>>(p);
        return cudaGetLastError();
    }
    auto* kernel = units == 8 ? cache_append_kernel<true, 128> : cache_append_kernel<true, 64>;
    const cudaError_t e = cudaFuncSetAttribute(
        kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSlots * 1024);
    if (e != cudaSuccess)
        return e;
    kernel<<<blocks, threads, kSlots * threads, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_cache_gather(const GatherParams& p, cudaStream_t stream)
{
    const unsigned blocks = (unsigned)((int64_t)p.pages * p.c.Hkv * p.c.B);
    if (p.c.e4m3)
        cache_gather_kernel<uint8_t><<<blocks, 128, 0, stream>>>(p);
    else
        cache_gather_kernel<__nv_bfloat16><<<blocks, 128, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace dfa
