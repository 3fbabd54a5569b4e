// dfa_paged.cu -- decoding attention over a paged cache, simple form: one block
// per query row, a warp per key in turn, fp32 throughout.
#include "dfa_serve.cuh"

namespace dfa {

namespace {

template <typename CELL, int D>
__global__ void __launch_bounds__(256) decode_paged_kernel(const __grid_constant__ PagedParams p)
{
    constexpr bool k8 = sizeof(CELL) == 1;
    constexpr int C = D / 32;
    __shared__ float s_m[8], s_l[8], s_o[8][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t i = blockIdx.x;
    const int32_t t = (int32_t)(i % p.T);
    i /= p.T;
    const int32_t hq = (int32_t)(i % p.Hq), b = (int32_t)(i / p.Hq), hk = hq / p.G;
    int32_t len, n;
    seq_rows(p.c, p.q_lens, p.T, b, len, n);
    if (t >= n)
        return;
    const int32_t keys = p.causal ? len - n + t + 1 : len;
    float q[C], o[C], m = -INFINITY, l = 0.f;
    const __nv_bfloat16* qr = (const __nv_bfloat16*)p.q.p + b * p.q.sb + hq * p.q.sh + t * p.q.sl;
    for (int c = 0; c < C; ++c) {
        q[c] = __bfloat162float(qr[lane * C + c]) * p.scale_log2;
        o[c] = 0.f;
    }
    for (int32_t j = warp; j < keys; j += 8) {
        const int32_t id = page_of(p.c, b, j / p.c.page);
        if (id < 0)
            continue;
        const int64_t at = (int64_t)id * p.c.page_stride +
                           ((int64_t)hk * p.c.page + j % p.c.page) * D + lane * C;
        float ks = 1.f, vs = 1.f, kf[C], vf[C];
        if (k8) {
            ks = p.c.k_scale[(int64_t)id * p.c.Hkv + hk];
            vs = p.c.v_scale[(int64_t)id * p.c.Hkv + hk];
            for (int c = 0; c < C; c += 2) {
                const float2 a = e4m3x2_float2(*(const uint16_t*)((const uint8_t*)p.c.k + at + c));
                const float2 w = e4m3x2_float2(*(const uint16_t*)((const uint8_t*)p.c.v + at + c));
                kf[c] = a.x, kf[c + 1] = a.y, vf[c] = w.x, vf[c + 1] = w.y;
            }
        } else {
            for (int c = 0; c < C; ++c) {
                kf[c] = __bfloat162float(((const __nv_bfloat16*)p.c.k)[at + c]);
                vf[c] = __bfloat162float(((const __nv_bfloat16*)p.c.v)[at + c]);
            }
        }
        float s = 0.f;
        for (int c = 0; c < C; ++c)
            s = fmaf(q[c], kf[c], s);
        for (int off = 16; off > 0; off >>= 1)
            s += __shfl_xor_sync(0xffffffffu, s, off);
        s *= ks;
        const float mn = fmaxf(m, s);
        const float alpha = mn == -INFINITY ? 1.f : exp2f(m - mn);
        const float pj = mn == -INFINITY ? exp2f(s) : exp2f(s - mn);
        l = l * alpha + pj;
        for (int c = 0; c < C; ++c)
            o[c] = o[c] * alpha + pj * vs * vf[c];
        m = mn;
    }
    if (lane == 0) {
        s_m[warp] = m;
        s_l[warp] = l;
    }
    for (int c = 0; c < C; ++c)
        s_o[warp][lane * C + c] = o[c];
    __syncthreads();
    float M = -INFINITY, L = 0.f, acc = 0.f;
    for (int w = 0; w < 8; ++w)
        M = fmaxf(M, s_m[w]);
    const int f = threadIdx.x;
    for (int w = 0; w < 8; ++w) {
        const float e = s_m[w] == -INFINITY ? (s_l[w] == 0.f ? 0.f : 1.f) : exp2f(s_m[w] - M);
        L += e * s_l[w];
        if (f < D)
            acc += e * s_o[w][f];
    }
    const int64_t row = ((int64_t)b * p.Hq + hq) * p.T + t;
    if (f < D) {
        const float r = L == 0.f ? 0.f : acc / L;
        if (p.o_fp32)
            ((float*)p.o)[row * D + f] = r;
        else
            ((__nv_bfloat16*)p.o)[row * D + f] = __float2bfloat16_rn(r);
    }
    if (f == 0)
        p.lse[row] = L == 0.f ? -INFINITY : (M == -INFINITY ? 0.f : M) * 0.69314718055994531f + logf(L);
}

}  // namespace

cudaError_t launch_decode_paged(const PagedParams& p, cudaStream_t stream)
{
    const unsigned blocks = (unsigned)((int64_t)p.c.B * p.Hq * p.T);
    if (p.c.e4m3) {
        if (p.c.d == 128)
            decode_paged_kernel<uint8_t, 128><<<blocks, 256, 0, stream>>>(p);
        else
            decode_paged_kernel<uint8_t, 64><<<blocks, 256, 0, stream>>>(p);
    } else {
        if (p.c.d == 128)
            decode_paged_kernel<__nv_bfloat16, 128><<<blocks, 256, 0, stream>>>(p);
        else
            decode_paged_kernel<__nv_bfloat16, 64><<<blocks, 256, 0, stream>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace dfa
