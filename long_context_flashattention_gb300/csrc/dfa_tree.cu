// dfa_tree.cu -- trees of drafted tokens over a paged cache: who sees whom and at which
// position, and attention of the tree's nodes over the cached rows.
#include "dfa_branch.h"
#include "dfa_serve.cuh"

namespace dfa {

namespace {

constexpr int kSiteParent = 103;  // of DFA_ERR_BOUNDS in DevStatus::where
constexpr float kLn2 = 0.69314718055994531f;

// One block per sequence.  sees[t] begins as node t itself and up[t] as its parent;
// a step adds what the node up[t] sees and moves up[t] to where that one points, so
// that after k steps the 2^k - 1 nearest ancestors are in.  (A word may be read
// while another thread adds to it: whatever it has more by then are ancestors too.)
__global__ void __launch_bounds__(1024) tree_plan_kernel(const __grid_constant__ TreePlanParams p)
{
    extern __shared__ uint32_t smem[];
    const int32_t T = p.T, W = p.words, b = blockIdx.x;
    volatile uint32_t* sees = smem;                    // [T][W]
    volatile int32_t* up = (int32_t*)(smem + T * W);   // [T]
    int32_t len, n;
    seq_rows(p.c, p.q_lens, T, b, len, n);
    for (int32_t t = threadIdx.x; t < n; t += blockDim.x) {
        int32_t parent = p.parents[(int64_t)b * T + t];
        if (parent < -1 || parent >= t) {
            cache_fault(p.c.status, kSiteParent, b);
            parent = -1;
        }
        up[t] = parent;
    }
    for (int32_t i = threadIdx.x; i < n * W; i += blockDim.x) {
        const int32_t t = i / W, w = i - t * W;
        sees[i] = t >> 5 == w ? 1u << (t & 31) : 0u;
    }
    __syncthreads();
    for (bool more = true; more;) {
        for (int32_t i = threadIdx.x; i < n * W; i += blockDim.x) {
            const int32_t t = i / W, w = i - t * W;
            const int32_t at = up[t];
            if (at >= 0 && w <= at >> 5)
                sees[i] = sees[i] | sees[at * W + w];
        }
        __syncthreads();
        // (T <= blockDim.x)
        int32_t next = -1;
        if ((int32_t)threadIdx.x < n) {
            const int32_t at = up[threadIdx.x];
            next = at >= 0 ? up[at] : -1;
        }
        __syncthreads();
        if ((int32_t)threadIdx.x < n)
            up[threadIdx.x] = next;
        more = __syncthreads_or(next >= 0);
    }
    for (int32_t i = threadIdx.x; i < n * W; i += blockDim.x)
        p.mask[(int64_t)b * T * W + i] = sees[i];
    for (int32_t t = threadIdx.x; t < n; t += blockDim.x) {
        int32_t seen = 0;
        for (int32_t w = 0; w <= t >> 5; ++w)
            seen += __popc(sees[t * W + w]);
        p.positions[(int64_t)b * T + t] = len - n + seen - 1;
    }
}

// One warp per query row: scores of 32 keys at a time, then their values.
template <int D, bool F8>
__global__ void __launch_bounds__(128) decode_tree_kernel(const __grid_constant__ TreeParams p)
{
    constexpr int V = D / 32;  // features of a lane
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= (int64_t)p.c.B * p.Hq * p.T)
        return;
    const int32_t t = row % p.T, hq = row / p.T % p.Hq, b = row / p.T / p.Hq, h = hq / p.G;
    int32_t len, n;
    seq_rows(p.c, p.q_lens, p.T, b, len, n);
    if (t >= n)
        return;
    const __nv_bfloat16* q =
        (const __nv_bfloat16*)p.q.p + b * p.q.sb + hq * p.q.sh + t * p.q.sl;
    const uint32_t* mask = p.mask + ((int64_t)b * p.T + t) * p.words;
    float m = -INFINITY, l = 0.f, o[V] = {};
    for (int32_t j0 = 0; j0 < len; j0 += 32) {
        const int32_t j = j0 + lane, node = j - (len - n);
        bool seen = j < len && (node < 0 || (mask[node >> 5] >> (node & 31) & 1));
        int32_t id = -1;
        if (seen) {
            id = page_of(p.c, b, j >> p.c.page_log2);
            seen = id >= 0;
        }
        const int64_t at = (int64_t)id * p.c.page_stride +
                           (((int64_t)h << p.c.page_log2) + (j & (p.c.page - 1))) * D;
        float x = -INFINITY, u = 1.f;
        if (seen) {
            float dot = 0.f;
            for (int f = 0; f < D; f += 2) {
                const float2 k = F8 ? e4m3x2_float2(*(const uint16_t*)((const uint8_t*)p.c.k + at + f))
                                    : __bfloat1622float2(*(const __nv_bfloat162*)((const __nv_bfloat16*)p.c.k + at + f));
                dot = fmaf(k.x, __bfloat162float(q[f]), dot);
                dot = fmaf(k.y, __bfloat162float(q[f + 1]), dot);
            }
            x = dot * p.scale_log2;
            if (F8) {
                x *= p.c.k_scale[(int64_t)id * p.c.Hkv + h];
                u = p.c.v_scale[(int64_t)id * p.c.Hkv + h];
            }
        }
        float mx = x;
        for (int i = 16; i > 0; i >>= 1)
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, i));
        if (!__any_sync(0xffffffffu, seen))
            continue;
        const float m2 = fmaxf(m, mx), f = m == -INFINITY ? 0.f : exp2f(m - m2);
        const float w = seen ? exp2f(x - m2) : 0.f;
        m = m2;
        l = l * f + w;
        for (int i = 0; i < V; ++i)
            o[i] *= f;
        for (int i = 0; i < 32; ++i) {
            if (!__shfl_sync(0xffffffffu, (int)seen, i))
                continue;
            const float wi = __shfl_sync(0xffffffffu, w * u, i);
            const int64_t ai = __shfl_sync(0xffffffffu, at, i);
            for (int v = 0; v < V; ++v)
                o[v] += wi * (F8 ? e4m3x2_float2(((const uint8_t*)p.c.v)[ai + lane * V + v]).x
                                 : __bfloat162float(((const __nv_bfloat16*)p.c.v)[ai + lane * V + v]));
        }
    }
    for (int i = 16; i > 0; i >>= 1)
        l += __shfl_xor_sync(0xffffffffu, l, i);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    for (int v = 0; v < V; ++v) {
        const int64_t to = row * D + lane * V + v;
        if (p.o_fp32)
            ((float*)p.o)[to] = o[v] * inv;
        else
            ((__nv_bfloat16*)p.o)[to] = __float2bfloat16(o[v] * inv);
    }
    if (lane == 0)
        p.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

}  // namespace

cudaError_t launch_tree_plan(const TreePlanParams& p, cudaStream_t stream)
{
    const int smem = p.T * (p.words + 1) * 4;
    const cudaError_t e = cudaFuncSetAttribute(
        tree_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
        kTreeMaxTokens * (kTreeMaxTokens / 32 + 1) * 4);
    if (e != cudaSuccess)
        return e;
    const int threads = min(1024, max(32, (p.T * min(p.words, 4) + 31) / 32 * 32));
    tree_plan_kernel<<<p.c.B, threads, smem, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_decode_tree(TreeParams& p, int num_sms, cudaStream_t stream)
{
    const unsigned blocks = (unsigned)(((int64_t)p.c.B * p.Hq * p.T + 3) / 4);
    if (p.c.e4m3)
        p.c.d == 128 ? decode_tree_kernel<128, true><<<blocks, 128, 0, stream>>>(p)
                     : decode_tree_kernel<64, true><<<blocks, 128, 0, stream>>>(p);
    else
        p.c.d == 128 ? decode_tree_kernel<128, false><<<blocks, 128, 0, stream>>>(p)
                     : decode_tree_kernel<64, false><<<blocks, 128, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace dfa
