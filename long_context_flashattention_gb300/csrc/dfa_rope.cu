// dfa_rope.cu -- rotary positions: rotation of query or key rows at explicit
// positions, either pair layout, part of the head, scaled frequencies, and the
// transposed rotation of the backward (Striped Attention Guide, "Preserving
// Rotary Position Embeddings": rotated inner products depend only on i - j).
//
// HBM-bound: every feature is read once and written once, three operations
// each.  What could bound it instead is the angles: a warp takes one token and
// several heads, its lanes compute the token's cos and sin once between them,
// and use them for all the heads.  Measured: 32 heads x 32768 x 128 in bf16 82 us,
// 6.5 TB/s (the copy rate is 6.8); 2 x 8 x 16381 x 128 in fp32 42.6 us, 6.3 TB/s.
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
    const SharedAngles<V, UNITS, kStep> angles(p.t, turns);
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
struct RopeRows {
    const RopeRowsParams& p;
    struct Token {
        uint32_t b, l;
        int32_t pos;
        bool ok;
    };
    __device__ __forceinline__ Token token(uint32_t i) const
    {
        const uint32_t b = i / (uint32_t)p.L, l = i - b * (uint32_t)p.L;
        return {b, l, p.positions ? __ldg(p.positions + i) : map_pos(p.map, (int32_t)l), true};
    }
    __device__ __forceinline__ const E* from(const Token& k, int32_t h) const
    {
        return (const E*)p.x.p + k.b * p.x.sb + k.l * p.x.sl + h * p.x.sh;
    }
    __device__ __forceinline__ E* to(const Token& k, int32_t h) const
    {
        return (E*)p.out.p + k.b * p.out.sb + k.l * p.out.sl + h * p.out.sh;
    }
    __device__ __forceinline__ bool turns(int32_t) const { return true; }
};

// Few heads: the lanes that heads do not take go to other tokens.  Measured (bf16,
// d 128, 2^20 rows of 1, 2, 4, 8 heads, us): 129, 99, 91, 89, where a warp a
// token takes 515, 272, 146, 101.  Two rows a lane and 4 blocks an SM; with sincospif,
// 141, 102, 92, 89, as against 2 and 3: 129, 101, 98, 95; 2 and 5 (spills): 168, 123,
// 113, 111; 4 and 2: 160, 129, 112, 106.  One head is bound by its own 64 angles a row
// (constant ones in their place: 89, 92, 92, 90).
constexpr int kFewBatch = 2;

template <typename E, int D, int G>
__global__ void __launch_bounds__(256, 4)
    rope_few_kernel(const __grid_constant__ RopeRowsParams p, uint32_t tokens)
{
    __shared__ uint64_t turns[64];
    if (threadIdx.x < 64)
        turns[threadIdx.x] = p.t.turn[threadIdx.x];
    __syncthreads();
    few_heads<E, D, G, kFewBatch>(p.t, turns, RopeRows<E>{p}, p.H, tokens,
                                  p.inverse ? -1.f : 1.f, blockIdx.x * 8 + (threadIdx.x >> 5),
                                  gridDim.x * 8);
}

template <typename E, int D>
cudaError_t launch(RopeRowsParams& p, int num_sms, cudaStream_t stream)
{
    constexpr int kStep = 32 / (D / (2 * Run<E>::V));
    const uint32_t rows = (uint32_t)(p.B * p.L);
    if (p.H <= 2 * kStep) {
        const int g = few_heads_group(p.H, kStep);
        const uint32_t each = (p.H > g ? kFewBatch / 2 : kFewBatch) * (kStep / g);
        const int blocks = (int)min((rows + 8 * each - 1) / (8 * each), num_sms * 8u);
        if (g == 1)
            rope_few_kernel<E, D, 1><<<blocks, 256, 0, stream>>>(p, rows);
        else if (g == 2)
            rope_few_kernel<E, D, kStep < 2 ? 1 : 2><<<blocks, 256, 0, stream>>>(p, rows);
        else if (g == 4)
            rope_few_kernel<E, D, kStep < 4 ? 1 : 4><<<blocks, 256, 0, stream>>>(p, rows);
        else
            rope_few_kernel<E, D, kStep < 8 ? 1 : 8><<<blocks, 256, 0, stream>>>(p, rows);
        return cudaGetLastError();
    }
    // Heads per warp: a warp computes its token's angles once for all of them, but
    // short inputs need the warps.  Measured (warps an SM to reach, 32 and 8; us): bf16
    // 32 heads x 512 4.9 3.7, x 2048 8.2 5.7, x 4096 10.2 9.4; 9 heads x 4096 7.8
    // 5.7; fp32 16 heads x 1024 5.8 4.1.  Twice as many heads a warp: 128 x 4096 bf16
    // 44.6 for 43.0, 32 x 4096 fp32 22.8 for 20.6; half as many: 32 x 2048 bf16 6.6.
    p.heads = 2 * kBatch * kStep;
    while (p.heads > kStep && rows * ((p.H + p.heads - 1) / p.heads) < num_sms * 8u)
        p.heads /= 2;
    const uint32_t head_items = (p.H + p.heads - 1) / p.heads;
    const uint32_t items = rows * head_items;
    const int blocks = (int)min((items + 7) / 8, num_sms * 8u);
    rope_rows_kernel<E, D><<<blocks, 256, 0, stream>>>(p, items, head_items);
    return cudaGetLastError();
}

}  // namespace

// (B * H * L is below 2^31.)
cudaError_t launch_rope_rows(RopeRowsParams& p, int fp32, int num_sms, cudaStream_t stream)
{
    if (fp32)
        return p.d == 128 ? launch<float, 128>(p, num_sms, stream)
                          : launch<float, 64>(p, num_sms, stream);
    return p.d == 128 ? launch<__nv_bfloat16, 128>(p, num_sms, stream)
                      : launch<__nv_bfloat16, 64>(p, num_sms, stream);
}

}  // namespace dfa
