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
// page and head and holds their features in registers in between: every row is
// read once.  The group keeps its rows' cos and sin in registers and goes
// through several heads with them.
//
// Row items (queries; K and V too in a bf16 cache, where rows are independent).
// A warp takes one token and several heads; its lanes compute the token's
// cos and sin once between them.
#include "dfa_serve.cuh"

namespace dfa {

namespace {

constexpr int kJobUnits = 1;  // 16-feature units of a page that a thread holds
constexpr int kBatch = 2;     // rows of an item in flight per lane

// codes of x / s; an infinity becomes NaN like a NaN, rather than the largest
// finite cell
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float inv)
{
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        y[i] = fabsf(x[i]) < INFINITY ? x[i] * inv : NAN;
    return make_uint2(e4m3x4(y[0], y[1], y[2], y[3]), e4m3x4(y[4], y[5], y[6], y[7]));
}

__device__ __forceinline__ float finite_abs(float x)
{
    const float y = fabsf(x);
    return y < INFINITY ? y : 0.f;  // NaN compares false
}

// Row items of a block.  Rows of a token: Hq queries, then (bf16 cache) Hkv keys
// and Hkv values.
template <bool F8, int D>
__device__ __forceinline__ void row_items(const AppendParams& p, uint32_t item, uint32_t stride)
{
    constexpr int UNITS = D / 16, kStep = 32 / UNITS;
    const int lane = threadIdx.x & 31;
    const int u = lane & (UNITS - 1), h_lane = lane / UNITS;
    const int32_t Hk = F8 ? 0 : p.c.Hkv, rows = p.Hq + 2 * Hk;
    const uint32_t per_token = (rows + p.item_heads - 1) / p.item_heads;
    int f0, f1;
    const bool turned = unit_runs<8>(p.t, D, u, f0, f1);
    const WarpAngles<8, UNITS> angles(p.t);
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
        int64_t cell = -1;  // first feature of the token's row of head 0
        if (!F8 && h1 > p.Hq) {
            const int32_t id = page_of(p.c, b, pos / p.c.page);
            if (id >= 0)
                cell = (int64_t)id * p.c.page_stride + (pos % p.c.page) * D;
        }
        float cs[8], sn[8];
        for (int32_t h = h0; h < h1; h += kBatch * kStep) {
            Run<__nv_bfloat16> r[kBatch][2];
            __nv_bfloat16* to[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int32_t hk = h + h_lane + k * kStep;
                to[k] = nullptr;
                if (hk >= h1)
                    continue;
                const __nv_bfloat16* from;
                if (F8 || hk < p.Hq) {
                    from = (const __nv_bfloat16*)p.q.p + b * p.q.sb + hk * p.q.sh + t * p.q.sl;
                    to[k] = (__nv_bfloat16*)p.q_out.p + b * p.q_out.sb + hk * p.q_out.sh +
                            t * p.q_out.sl;
                } else {
                    if (cell < 0)
                        continue;
                    const bool is_v = hk >= p.Hq + Hk;
                    const int32_t hc = hk - p.Hq - (is_v ? Hk : 0);
                    const Rows& src = is_v ? p.v : p.k;
                    from = (const __nv_bfloat16*)src.p + b * src.sb + hc * src.sh + t * src.sl;
                    to[k] = (__nv_bfloat16*)(is_v ? p.c.v : p.c.k) + cell +
                            (int64_t)hc * p.c.page * D;
                }
                r[k][0].load(from + f0);
                r[k][1].load(from + f1);
            }
            if (h == h0 && p.t.half && h0 < p.Hq + Hk)  // not for values alone
                angles.at(pos, 1.f, cs, sn);
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                if (!to[k])
                    continue;
                if (turned && h + h_lane + k * kStep < p.Hq + Hk) {
                    float a[8], c[8];
                    r[k][0].get(a);
                    r[k][1].get(c);
                    unit_rotate<8>(p.t, cs, sn, a, c);
                    r[k][0].set(a);
                    r[k][1].set(c);
                }
                r[k][0].store(to[k] + f0);
                r[k][1].store(to[k] + f1);
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

// One page job: K or V rows of one page, job_heads heads.  Every thread of the
// group takes the same way through it.
template <int D>
__device__ __forceinline__ void page_job(const AppendParams& p, uint32_t job, int group,
                                         int thread, const uint64_t* turn, float (*warp_max)[32])
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
    int32_t len, n;
    seq_rows(p.c, p.new_lens, p.T, b, len, n);
    const int32_t first = len - n;                 // first new row
    const int32_t pg = first / p.c.page + ip;      // page of the sequence
    const int32_t lo = max(first, pg * p.c.page);  // rows [lo, hi) are new
    const int32_t hi = min(len, (pg + 1) * p.c.page);
    if (lo >= hi)
        return;
    const int32_t id = page_of(p.c, b, pg);
    if (id < 0)
        return;
    const int threads = p.job_threads, warps = threads / 32;
    const Rows& src = is_v ? p.v : p.k;
    float* scales = (is_v ? p.c.v_scale : p.c.k_scale) + (int64_t)id * p.c.Hkv;
    const int32_t there = lo - pg * p.c.page;  // rows of the page stored before
    const int32_t u = thread & (UNITS - 1);    // threads is a multiple of UNITS
    int f0, f1;
    const bool turned = unit_runs<8>(p.t, D, u, f0, f1) && !is_v;
    float cs[kJobUnits][8], sn[kJobUnits][8];
    const int32_t h1 = min(h0 + p.job_heads, p.c.Hkv);
    for (int32_t h = h0; h < h1; ++h) {
        const __nv_bfloat16* x =
            (const __nv_bfloat16*)src.p + b * src.sb + h * src.sh - (int64_t)first * src.sl;
        uint8_t* cells = (uint8_t*)(is_v ? p.c.v : p.c.k) + (int64_t)id * p.c.page_stride +
                         (int64_t)h * p.c.page * D;
        Run<__nv_bfloat16> raw[kJobUnits][2];
#pragma unroll
        for (int k = 0; k < kJobUnits; ++k) {
            const int32_t row = lo + (thread + k * threads) / UNITS;
            if (row < hi) {
                raw[k][0].load(x + row * src.sl + f0);
                raw[k][1].load(x + row * src.sl + f1);
            }
        }
        const float old = there > 0 ? scales[h] : 0.f;
        if (h == h0 && turned)
#pragma unroll
            for (int k = 0; k < kJobUnits; ++k) {
                const int32_t row = lo + (thread + k * threads) / UNITS;
                if (row < hi)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        pair_angle(turn[unit_pair<8>(p.t, u, j)], p.t.gain, row, 1.f, cs[k][j],
                                   sn[k][j]);
            }
        float a[kJobUnits][8], c[kJobUnits][8], amax = 0.f;
#pragma unroll
        for (int k = 0; k < kJobUnits; ++k) {
            if (lo + (thread + k * threads) / UNITS >= hi)
                continue;
            raw[k][0].get(a[k]);
            raw[k][1].get(c[k]);
            if (turned)
                unit_rotate<8>(p.t, cs[k], sn[k], a[k], c[k]);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                amax = fmaxf(amax, fmaxf(finite_abs(a[k][j]), finite_abs(c[k][j])));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if (warps > 1) {
            // two sets of maxima, so that one barrier a head is enough
            float* wm = warp_max[(h & 1) * 16 + group];
            if ((thread & 31) == 0)
                wm[thread >> 5] = amax;
            group_sync(group, threads);
            for (int w = 0; w < warps; ++w)
                amax = fmaxf(amax, wm[w]);
        }
        const float s = fmaxf(old, pow2_scale(amax));
        const float inv = 1.f / s;  // exact: a power of two (or a scale of the caller's)
        if (s > old && there > 0) {
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
        if (s != old) {
            // everyone has read the old scale (the barrier, or the warp's shuffles)
            if (warps <= 1)
                __syncwarp();
            if (thread == 0)
                scales[h] = s;
        }
#pragma unroll
        for (int k = 0; k < kJobUnits; ++k) {
            const int32_t row = lo + (thread + k * threads) / UNITS;
            if (row < hi) {
                uint8_t* cell = cells + (row - pg * p.c.page) * D;
                *reinterpret_cast<uint2*>(cell + f0) = codes8(a[k], inv);
                *reinterpret_cast<uint2*>(cell + f1) = codes8(c[k], inv);
            }
        }
    }
}

template <bool F8, int D>
__global__ void __launch_bounds__(F8 ? 1024 : 256, F8 ? 1 : 3)
    cache_append_kernel(const __grid_constant__ AppendParams p)
{
    if (F8 && (int32_t)blockIdx.x < p.job_blocks) {
        __shared__ float warp_max[32][32];
        __shared__ uint64_t turn[64];  // lanes read different entries: not from the parameters
        if (threadIdx.x < 64)
            turn[threadIdx.x] = p.t.turn[threadIdx.x];
        __syncthreads();
        const int groups = blockDim.x / p.job_threads;
        const int group = threadIdx.x / p.job_threads;
        const uint32_t job = blockIdx.x * groups + group;
        if (job < p.jobs)
            page_job<D>(p, job, group, threadIdx.x - group * p.job_threads, turn, warp_max);
        return;
    }
    const int warps = blockDim.x >> 5;
    row_items<F8, D>(p, (blockIdx.x - p.job_blocks) * warps + (threadIdx.x >> 5),
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

// Blocks that have work at once are some 8 an SM; below that a job or an item
// takes as few heads as it can, above it as many as pay (angles are computed
// once per job or item).
cudaError_t launch_cache_append(AppendParams& p, int num_sms, cudaStream_t stream)
{
    const int units = p.c.d / 16, step = 32 / units;
    const int64_t tokens = (int64_t)p.c.B * p.T;
    int threads = 256;
    if (p.c.e4m3) {
        const int rows = min(p.T, p.c.page);
        p.job_threads = 32;
        while (p.job_threads * kJobUnits < rows * units)
            p.job_threads *= 2;
        threads = max(threads, p.job_threads);
        const int64_t pages = (int64_t)p.c.B * 2 * p.pages;  // of one head
        p.job_heads = 8;
        while (p.job_heads > 1 &&
               pages * ((p.c.Hkv + p.job_heads - 1) / p.job_heads) * p.job_threads <
                   (int64_t)num_sms * 2048)
            p.job_heads /= 2;
        p.jobs = (uint32_t)(pages * ((p.c.Hkv + p.job_heads - 1) / p.job_heads));
        const int groups = threads / p.job_threads;
        p.job_blocks = (int32_t)((p.jobs + groups - 1) / groups);
    }
    const int rows = p.Hq + (p.c.e4m3 ? 0 : 2 * p.c.Hkv);
    int64_t item_blocks = 0;
    if (rows > 0) {
        p.item_heads = 16 * kBatch * step;
        while (p.item_heads > step &&
               tokens * ((rows + p.item_heads - 1) / p.item_heads) < (int64_t)num_sms * 64)
            p.item_heads /= 2;
        p.items = (uint32_t)(tokens * ((rows + p.item_heads - 1) / p.item_heads));
        item_blocks = min((p.items + threads / 32 - 1) / (threads / 32), num_sms * 64u);
    }
    const unsigned blocks = (unsigned)(p.job_blocks + item_blocks);
    if (p.c.e4m3) {
        if (units == 8)
            cache_append_kernel<true, 128><<<blocks, threads, 0, stream>>>(p);
        else
            cache_append_kernel<true, 64><<<blocks, threads, 0, stream>>>(p);
    } else {
        if (units == 8)
            cache_append_kernel<false, 128><<<blocks, threads, 0, stream>>>(p);
        else
            cache_append_kernel<false, 64><<<blocks, threads, 0, stream>>>(p);
    }
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
