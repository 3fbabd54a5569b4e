// dfa_cache.cu -- the paged key/value cache: append of new rows (keys rotated,
// both quantised to 8 bits with a power-of-two scale per page and head, or kept
// in bf16) together with the rotation of the queries that go with them, and
// gather of cached rows into contiguous bf16.
//
// Both are HBM-bound for long inputs (a few operations per feature) and bound
// by the chain of dependent loads (length -> page -> scale -> rows) for one
// token.  Append: one block per (sequence, K or V, head, page), because a page's
// scale needs the largest value of all its rows before the first is stored; a
// block holds its rows' features in registers between the two, so every row is
// read once.
#include "dfa_serve.cuh"

namespace dfa {

namespace {

constexpr int kUnitsPerThread = 4;  // 16-feature units a thread holds: 64 fp32

__device__ __forceinline__ void store_cells(__nv_bfloat16* row, int f0, int f1, const float (&a)[8],
                                            const float (&b)[8], float)
{
    Raw8<__nv_bfloat16> r;
    r.set(a);
    r.store(row + f0);
    r.set(b);
    r.store(row + f1);
}

// codes of x / s; an infinity becomes NaN like a NaN, rather than the largest
// finite cell
__device__ __forceinline__ void store_cells(uint8_t* row, int f0, int f1, const float (&a)[8],
                                            const float (&b)[8], float inv)
{
    float x[8], y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[i] = fabsf(a[i]) < INFINITY ? a[i] * inv : NAN;
        y[i] = fabsf(b[i]) < INFINITY ? b[i] * inv : NAN;
    }
    *reinterpret_cast<uint2*>(row + f0) =
        make_uint2(e4m3x4(x[0], x[1], x[2], x[3]), e4m3x4(x[4], x[5], x[6], x[7]));
    *reinterpret_cast<uint2*>(row + f1) =
        make_uint2(e4m3x4(y[0], y[1], y[2], y[3]), e4m3x4(y[4], y[5], y[6], y[7]));
}

__device__ __forceinline__ float finite_abs(float x)
{
    const float y = fabsf(x);
    return y < INFINITY ? y : 0.f;  // NaN compares false
}

// Queries: one warp per (sequence, token, 32/units heads).
__device__ __forceinline__ void append_queries(const AppendParams& p, int64_t item)
{
    const int units = p.c.d / 16;
    const int lane = threadIdx.x & 31;
    const int u = lane & (units - 1), per = 32 / units;
    const int32_t head_items = (p.Hq + per - 1) / per;
    const int64_t row = item / head_items;
    const int32_t h = (int32_t)(item - row * head_items) * per + lane / units;
    const int32_t b = (int32_t)(row / p.T);
    if (b >= p.c.B)
        return;
    const int32_t t = (int32_t)(row - (int64_t)b * p.T);
    int32_t len, n;
    seq_rows(p.c, p.new_lens, p.T, b, len, n);
    if (t >= n)
        return;
    int f0, f1;
    unit_runs(p.t, u, f0, f1);
    const bool turned = u < p.t.units;
    float cs[8], sn[8];
    if (turned)
        unit_angles(p.t, u, len - n + t, 1.f, cs, sn);
    rotate_heads<1>(p.t, turned, cs, sn,
                    (const __nv_bfloat16*)p.q.p + b * p.q.sb + (int64_t)t * p.q.sl, p.q.sh,
                    (__nv_bfloat16*)p.q_out.p + b * p.q_out.sb + (int64_t)t * p.q_out.sl,
                    p.q_out.sh, f0, f1, h, min(h + 1, p.Hq), 1);
}

// CELL: uint8_t (e4m3) or __nv_bfloat16
template <typename CELL>
__global__ void __launch_bounds__(256) cache_append_kernel(const __grid_constant__ AppendParams p)
{
    constexpr bool k8 = sizeof(CELL) == 1;
    if (blockIdx.x >= p.kv_blocks) {
        const int warps = blockDim.x >> 5;
        append_queries(p, (int64_t)(blockIdx.x - p.kv_blocks) * warps + (threadIdx.x >> 5));
        return;
    }
    // page innermost: consecutive blocks read consecutive rows of one head
    int32_t i = blockIdx.x;
    const int32_t ip = i % p.pages;
    i /= p.pages;
    const int32_t h = i % p.c.Hkv;
    i /= p.c.Hkv;
    const int32_t is_v = i & 1, b = i >> 1;
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
    const int32_t d = p.c.d, units = d / 16;
    CELL* cells = (CELL*)(is_v ? p.c.v : p.c.k) + (int64_t)id * p.c.page_stride +
                  (int64_t)h * p.c.page * d;
    const Rows& src = is_v ? p.v : p.k;
    const __nv_bfloat16* x = (const __nv_bfloat16*)src.p + b * src.sb + h * src.sh -
                             (int64_t)first * src.sl;
    float a[kUnitsPerThread][8], c[kUnitsPerThread][8];
    float amax = 0.f;
#pragma unroll
    for (int k = 0; k < kUnitsPerThread; ++k) {
        const int32_t idx = threadIdx.x + k * blockDim.x;
        const int32_t row = lo + idx / units, u = idx % units;
        if (row < hi) {
            int f0, f1;
            unit_runs(p.t, u, f0, f1);
            Raw8<__nv_bfloat16> r0, r1;
            r0.load(x + row * src.sl + f0);
            r1.load(x + row * src.sl + f1);
            r0.get(a[k]);
            r1.get(c[k]);
        }
    }
#pragma unroll
    for (int k = 0; k < kUnitsPerThread; ++k) {
        const int32_t idx = threadIdx.x + k * blockDim.x;
        const int32_t row = lo + idx / units, u = idx % units;
        if (row >= hi)
            continue;
        if (!is_v && u < p.t.units) {
            float cs[8], sn[8];
            unit_angles(p.t, u, row, 1.f, cs, sn);
            unit_rotate(p.t, cs, sn, a[k], c[k]);
        }
        if (k8) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                amax = fmaxf(amax, fmaxf(finite_abs(a[k][j]), finite_abs(c[k][j])));
        }
    }
    float inv = 1.f;
    if (k8) {
        __shared__ float warp_max[8];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if ((threadIdx.x & 31) == 0)
            warp_max[threadIdx.x >> 5] = amax;
        float* scale = (is_v ? p.c.v_scale : p.c.k_scale) + (int64_t)id * p.c.Hkv + h;
        const int32_t there = lo - pg * p.c.page;  // rows of the page stored before
        const float old = there > 0 ? *scale : 0.f;
        __syncthreads();
        for (int w = 0; w < (blockDim.x >> 5); ++w)
            amax = fmaxf(amax, warp_max[w]);
        const float s = fmaxf(old, pow2_scale(amax));
        inv = 1.f / s;  // exact: a power of two (or a scale of the caller's)
        if (s > old && there > 0) {
            // raise the rows that are there to the new scale: exact but for
            // cells that become subnormal
            const float f = old * inv;
            for (int32_t v = threadIdx.x; v < there * d / 16; v += blockDim.x) {
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
        if (threadIdx.x == 0 && s != old)
            *scale = s;
    }
#pragma unroll
    for (int k = 0; k < kUnitsPerThread; ++k) {
        const int32_t idx = threadIdx.x + k * blockDim.x;
        const int32_t row = lo + idx / units, u = idx % units;
        if (row < hi) {
            int f0, f1;
            unit_runs(p.t, u, f0, f1);
            store_cells(cells + (row - pg * p.c.page) * d, f0, f1, a[k], c[k], inv);
        }
    }
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

cudaError_t launch_cache_append(const AppendParams& p, int64_t q_items, cudaStream_t stream)
{
    // as many threads as hold a page in registers
    const int threads = max(32, p.c.page * p.c.d / 16 / kUnitsPerThread);
    const int warps = threads / 32;
    const unsigned blocks = (unsigned)(p.kv_blocks + (q_items + warps - 1) / warps);
    if (p.c.e4m3)
        cache_append_kernel<uint8_t><<<blocks, threads, 0, stream>>>(p);
    else
        cache_append_kernel<__nv_bfloat16><<<blocks, threads, 0, stream>>>(p);
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
