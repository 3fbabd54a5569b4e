// dfa_rope.cu -- rotary positions: rotation of query or key rows at explicit
// positions, either pair layout, part of the head, scaled frequencies, and the
// transposed rotation of the backward (Striped Attention Guide, "Preserving
// Rotary Position Embeddings": rotated inner products depend only on i - j).
//
// HBM-bound: every feature is read once and written once, three operations
// each.  What could bound it instead is the angles, 8 per 16-feature unit of a
// token: a warp takes one token and several heads, so a lane computes its
// unit's angles once and uses them for all its heads.
#include "dfa_serve.cuh"

namespace dfa {

// One warp per item = (batch, token, `heads` heads); lane = (head, unit).
template <typename E>
__global__ void __launch_bounds__(256) rope_rows_kernel(const __grid_constant__ RopeRowsParams p,
                                                        int64_t items, int32_t head_items)
{
    const int units = p.d / 16;
    const int lane = threadIdx.x & 31;
    const int u = lane & (units - 1);
    const int h_lane = lane / units, h_step = 32 / units;
    int f0, f1;
    unit_runs(p.t, u, f0, f1);
    const bool turned = u < p.t.units;
    // features that pass through are already there when the call works in place
    if (!turned && p.x.p == p.out.p)
        return;
    for (int64_t it = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); it < items;
         it += (int64_t)gridDim.x * 8) {
        const int64_t row = it / head_items;
        const int32_t h0 = (int32_t)(it - row * head_items) * p.heads;
        const int32_t b = (int32_t)(row / p.L);
        const int64_t l = row - (int64_t)b * p.L;
        float cs[8], sn[8];
        if (turned) {
            const int32_t pos = p.positions ? __ldg(p.positions + row) : map_pos(p.map, (int32_t)l);
            unit_angles(p.t, u, pos, p.inverse ? -1.f : 1.f, cs, sn);
        }
        const E* x = (const E*)p.x.p + b * p.x.sb + l * p.x.sl;
        E* out = (E*)p.out.p + b * p.out.sb + l * p.out.sl;
        const int32_t h1 = min(h0 + p.heads, p.H);
        rotate_heads<4>(p.t, turned, cs, sn, x, p.x.sh, out, p.out.sh, f0, f1, h0 + h_lane, h1,
                        h_step);
    }
}

cudaError_t launch_rope_rows(const RopeRowsParams& p, int fp32, int num_sms, cudaStream_t stream)
{
    const int32_t head_items = (p.H + p.heads - 1) / p.heads;
    const int64_t items = (int64_t)p.B * p.L * head_items;
    int64_t blocks = (items + 7) / 8;
    const int64_t cap = (int64_t)num_sms * 8;
    if (blocks > cap)
        blocks = cap;
    if (fp32)
        rope_rows_kernel<float><<<(int)blocks, 256, 0, stream>>>(p, items, head_items);
    else
        rope_rows_kernel<__nv_bfloat16><<<(int)blocks, 256, 0, stream>>>(p, items, head_items);
    return cudaGetLastError();
}

}  // namespace dfa
