// dfa_tree.cu -- the plan of trees of drafted tokens: who sees whom, and at which position.
#include "dfa_branch.h"
#include "dfa_serve.cuh"

namespace dfa {

namespace {

constexpr int kSiteParent = 103;  // of DFA_ERR_BOUNDS in DevStatus::where

// One block per sequence, nodes in groups of 32.  First, every group by a warp of its own:
// which of a node's ancestors are in its group, and the nearest one before the group, by
// doubling how far up the lanes know.  Then group after group: a node sees what that one
// sees, and in its own group's word the former.  A warp takes four nodes, a lane a word;
// of node t only words up to t / 32 are kept.
//
// Bound by the output and by the groups' order for many deep trees (256 of 1024 nodes, 34 MB:
// 15.5 us, other trees each time 17; one doubling of whole rows per step took 107), by the
// chain of loads for small ones (64 of up to 60 nodes: 2.5 us).
__global__ void __launch_bounds__(256) tree_plan_kernel(const __grid_constant__ TreePlanParams p)
{
    extern __shared__ uint32_t sees[];            // group g: 32 nodes of g + 1 words
    // of a node: the nearest ancestor before its group, as the place of its words and its
    // group (<< 16), or -1; the ancestors in the group
    __shared__ __align__(16) int32_t from[kTreeMaxTokens];
    __shared__ __align__(16) uint32_t own[kTreeMaxTokens];
    const int32_t T = p.T, W = p.words, b = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int32_t len, n;
    seq_rows(p.c, p.q_lens, T, b, len, n);
    const int32_t groups = (n + 31) / 32;
    for (int32_t g = warp; g < groups; g += 8) {
        const int32_t t = 32 * g + lane;
        int32_t parent = t < n ? p.parents[(int64_t)b * T + t] : -1;
        if (parent < -1 || parent >= t) {
            cache_fault(p.c.status, kSiteParent, b);
            parent = -1;
        }
        const bool inside = parent >= 32 * g;
        int32_t up = inside ? parent - 32 * g : lane;  // (a node without one here: itself)
        uint32_t bits = 1u << lane;
#pragma unroll
        for (int i = 0; i < 5; ++i) {
            bits |= __shfl_sync(0xffffffffu, bits, up);
            up = __shfl_sync(0xffffffffu, up, up);
        }
        // (up: the ancestor here whose parent is not)
        const int32_t f = __shfl_sync(0xffffffffu, parent, up), fg = f >> 5;
        from[t] = f < 0 ? -1 : (fg + 1) * (16 * fg + (f & 31)) | fg << 16;
        own[t] = bits;
    }
    __syncthreads();
    const int32_t t4 = warp * 4;  // the warp's nodes of a group
    uint32_t* out = p.mask + ((int64_t)b * T + t4) * W + lane;
    int4 f4 = *reinterpret_cast<const int4*>(from + t4);
    uint4 o4 = *reinterpret_cast<const uint4*>(own + t4);
    for (int32_t g = 0; g < groups; ++g, out += 32 * W) {
        const int32_t f[4] = {f4.x, f4.y, f4.z, f4.w};
        const uint32_t o[4] = {o4.x, o4.y, o4.z, o4.w};
        uint32_t word[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            word[k] = lane == g ? o[k] : 0u;
            if (f[k] >= 0 && lane <= f[k] >> 16)
                word[k] = sees[(f[k] & 0xffff) + lane];
        }
        if (lane <= g) {
            uint32_t* to = sees + (g + 1) * (16 * g + t4) + lane;
#pragma unroll
            for (int k = 0; k < 4; ++k, to += g + 1)
                *to = word[k];
        }
        const int32_t t = 32 * g + t4;
        if (g + 1 < groups) {
            f4 = *reinterpret_cast<const int4*>(from + t + 32);
            o4 = *reinterpret_cast<const uint4*>(own + t + 32);
        }
        __syncthreads();  // (then the next group; what is left of this one beside it)
        int32_t depth = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (lane < W && t + k < n)
                out[k * W] = word[k];
            const int32_t bits = __reduce_add_sync(0xffffffffu, __popc(word[k]));
            depth = lane == k ? bits : depth;
        }
        if (lane < 4 && t + lane < n)
            p.positions[(int64_t)b * T + t + lane] = len - n + depth - 1;
    }
}

}  // namespace

cudaError_t launch_tree_plan(const TreePlanParams& p, cudaStream_t stream)
{
    const int groups = p.words;
    const int most = 16 * 32 * 33 * 4, smem = groups > 1 ? 16 * groups * (groups + 1) * 4 : 128;
    const cudaError_t e = cudaFuncSetAttribute(
        tree_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess)
        return e;
    tree_plan_kernel<<<p.c.B, 256, smem, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace dfa
