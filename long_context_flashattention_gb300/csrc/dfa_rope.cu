// dfa_rope.cu -- rotary positions: rotation of query or key rows at explicit
// positions, either pair layout, part of the head, scaled frequencies, and the
// transposed rotation of the backward (Striped Attention Guide, "Preserving
// Rotary Position Embeddings": rotated inner products depend only on i - j).
//
// HBM-bound: every feature is read once and written once, three operations
// each.  What could bound it instead is the angles: a warp takes one token and
// several heads, its lanes compute the token's cos and sin once between them,
// and use them for all the heads.
#include "dfa_serve.cuh"

namespace dfa {

namespace {

// Rows in flight per lane.  Measured (bf16 32 heads x 32768 x 128, fp32 2 x 8 x
// 16381 x 128, us; blocks an SM by registers): 4 rows and 3 blocks 84.4, 42.8;
// 4 and 2 82.1, 45.1; 2 and 4 87.6, 43.8.
constexpr int kBatch = 4;

// One warp per item = (batch, token, `heads` heads); lane = (head, unit).
template <typename E, int D>
__global__ void __launch_bounds__(256, sizeof(E) == 2 ? 2 : 3)
    rope_rows_kernel(const __grid_constant__ RopeRowsParams p, uint32_t items, uint32_t head_items)
{
    constexpr int V = Run<E>::V, UNITS = D / (2 * V), kStep = 32 / UNITS;
    const int lane = threadIdx.x & 31;
    const int u = lane & (UNITS - 1), h_lane = lane / UNITS;
    int f0, f1;
    const bool turned = unit_runs<V>(p.t, D, u, f0, f1);
    // features that pass through are already there when the call works in place
    const bool move = turned || p.x.p != p.out.p;
    __shared__ uint64_t turns[64];
    if (threadIdx.x < 64)
        turns[threadIdx.x] = p.t.turn[threadIdx.x];
    __syncthreads();
    const WarpAngles<V, UNITS> angles(p.t, turns);
    for (uint32_t it = blockIdx.x * 8 + (threadIdx.x >> 5); it < items; it += gridDim.x * 8) {
        const uint32_t row = it / head_items;
        const int32_t h0 = (int32_t)(it - row * head_items) * p.heads;
        const uint32_t b = row / (uint32_t)p.L, l = row - b * (uint32_t)p.L;
        const int32_t pos = p.positions ? __ldg(p.positions + row) : map_pos(p.map, (int32_t)l);
        const E* x = (const E*)p.x.p + b * p.x.sb + l * p.x.sl;
        E* out = (E*)p.out.p + b * p.out.sb + l * p.out.sl;
        const int32_t h1 = min(h0 + p.heads, p.H);
        float cs[V], sn[V];
        for (int32_t h = h0; h < h1; h += kBatch * kStep) {
            Run<E> r[kBatch][2];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int32_t hk = h + h_lane + k * kStep;
                if (move && hk < h1) {
                    r[k][0].load(x + hk * p.x.sh + f0);
                    r[k][1].load(x + hk * p.x.sh + f1);
                }
            }
            if (h == h0)  // while the first rows are on their way
                angles.at(pos, p.inverse ? -1.f : 1.f, cs, sn);
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int32_t hk = h + h_lane + k * kStep;
                if (move && hk < h1) {
                    if (turned) {
                        float a[V], c[V];
                        r[k][0].get(a);
                        r[k][1].get(c);
                        unit_rotate<V>(p.t, cs, sn, a, c);
                        r[k][0].set(a);
                        r[k][1].set(c);
                    }
                    r[k][0].store(out + hk * p.out.sh + f0);
                    r[k][1].store(out + hk * p.out.sh + f1);
                }
            }
        }
    }
}

template <typename E>
void launch(const RopeRowsParams& p, int blocks, uint32_t items, uint32_t head_items,
            cudaStream_t stream)
{
    if (p.d == 128)
        rope_rows_kernel<E, 128><<<blocks, 256, 0, stream>>>(p, items, head_items);
    else
        rope_rows_kernel<E, 64><<<blocks, 256, 0, stream>>>(p, items, head_items);
}

}  // namespace

// Heads per warp: a warp computes its token's angles once for all of them, but
// short inputs need the warps.  (B * H * L is below 2^31.)
cudaError_t launch_rope_rows(RopeRowsParams& p, int fp32, int num_sms, cudaStream_t stream)
{
    const int step = 32 / (p.d / (fp32 ? 8 : 16));
    const uint32_t rows = (uint32_t)(p.B * p.L);
    p.heads = 4 * kBatch * step;
    while (p.heads > step && rows * ((p.H + p.heads - 1) / p.heads) < num_sms * 32u)
        p.heads /= 2;
    const uint32_t head_items = (p.H + p.heads - 1) / p.heads;
    const uint32_t items = rows * head_items;
    const int blocks = (int)min((items + 7) / 8, num_sms * 8u);
    if (fp32)
        launch<float>(p, blocks, items, head_items, stream);
    else
        launch<__nv_bfloat16>(p, blocks, items, head_items, stream);
    return cudaGetLastError();
}

}  // namespace dfa
