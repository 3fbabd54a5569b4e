// dfa_tree.cu -- the plan of trees of drafted tokens: who sees whom, and at which position.
#include "dfa_branch.h"
#include "dfa_serve.cuh"

namespace dfa {

namespace {

constexpr int kSiteParent = 103;  // of DFA_ERR_BOUNDS in DevStatus::where

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

}  // namespace dfa
