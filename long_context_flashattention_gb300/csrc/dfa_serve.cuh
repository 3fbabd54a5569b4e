// dfa_serve.cuh -- device helpers of the rotary and paged-cache kernels:
// checked lengths and pages, the rotation of a 16-feature unit, 8-bit cells.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "dfa_ptx.cuh"
#include "dfa_serve.h"

namespace dfa {

// Sites of DFA_ERR_BOUNDS in DevStatus::where.
constexpr int kSiteSeqLen = 100, kSiteNewLen = 101, kSitePage = 102;

__device__ __forceinline__ void cache_fault(DevStatus* st, int site, int detail)
{
    if (atomicCAS(&st->code, 0, kStatusBounds) == 0) {
        st->where = site;
        st->detail = detail;
    }
}

// Rows of sequence b, and how many of them are new (or queried).  A length out
// of range is reported and makes the sequence empty.
__device__ __forceinline__ void seq_rows(const CacheView& c, const int32_t* new_lens, int32_t T,
                                         int32_t b, int32_t& len, int32_t& n)
{
    len = __ldg(c.seq_lens + b);
    n = new_lens ? __ldg(new_lens + b) : T;
    if (len < 0 || len > (int64_t)c.max_pages * c.page) {
        cache_fault(c.status, kSiteSeqLen, b);
        len = n = 0;
    } else if (n < 0 || n > T || n > len) {
        cache_fault(c.status, kSiteNewLen, b);
        len = n = 0;
    }
}

// Page number of rows [i*page, (i+1)*page) of sequence b; -1 (reported) when
// it is out of range.  i < max_pages.
__device__ __forceinline__ int32_t page_of(const CacheView& c, int32_t b, int32_t i)
{
    const int32_t id = __ldg(c.table + (int64_t)b * c.max_pages + i);
    if (id < 0 || id >= c.npages) {
        cache_fault(c.status, kSitePage, b);
        return -1;
    }
    return id;
}

// ---------------------------------------------------------------------------
// rotation: a unit is 8 feature pairs (16 features); unit u < units holds the
// pairs 8u..8u+7.  Its features are two runs of 8: in the half layout 8u.. and
// half + 8u.., else 16u.. and 16u + 8...
// ---------------------------------------------------------------------------
__device__ __forceinline__ void unit_runs(const RopeTable& t, int u, int& f0, int& f1)
{
    const bool apart = t.half_layout && u < t.units;
    f0 = apart ? 8 * u : 16 * u;
    f1 = apart ? t.half + 8 * u : 16 * u + 8;
}

// cos and sin (gain included) of the unit's pairs at a position.  The top 32
// bits of the phase are the angle in half turns times 2^31.
__device__ __forceinline__ void unit_angles(const RopeTable& t, int u, int32_t pos, float sign,
                                            float (&cs)[8], float (&sn)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint64_t ph = (uint64_t)(int64_t)pos * t.turn[8 * u + i];
        sincospif((float)(int32_t)(ph >> 32) * 4.656612873077393e-10f, &sn[i], &cs[i]);
        cs[i] *= t.gain;
        sn[i] *= t.gain * sign;
    }
}

// a, b: the unit's two runs
__device__ __forceinline__ void unit_rotate(const RopeTable& t, const float (&cs)[8],
                                            const float (&sn)[8], float (&a)[8], float (&b)[8])
{
    if (t.half_layout) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x = a[i], y = b[i];
            a[i] = x * cs[i] - y * sn[i];
            b[i] = x * sn[i] + y * cs[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x = a[2 * i], y = a[2 * i + 1], z = b[2 * i], w = b[2 * i + 1];
            a[2 * i] = x * cs[i] - y * sn[i];
            a[2 * i + 1] = x * sn[i] + y * cs[i];
            b[2 * i] = z * cs[i + 4] - w * sn[i + 4];
            b[2 * i + 1] = z * sn[i + 4] + w * cs[i + 4];
        }
    }
}

// Eight features: as they lie in memory, and as fp32.  (Plain loads: a call may
// work in place.)
template <typename E>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
    uint4 w;
    __device__ __forceinline__ void load(const __nv_bfloat16* p)
    {
        w = *reinterpret_cast<const uint4*>(p);
    }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const
    {
        *reinterpret_cast<uint4*>(p) = w;
    }
    __device__ __forceinline__ void get(float (&f)[8]) const
    {
        f[0] = bf16lo(w.x), f[1] = bf16hi(w.x), f[2] = bf16lo(w.y), f[3] = bf16hi(w.y);
        f[4] = bf16lo(w.z), f[5] = bf16hi(w.z), f[6] = bf16lo(w.w), f[7] = bf16hi(w.w);
    }
    __device__ __forceinline__ void set(const float (&f)[8])
    {
        w = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                       pack_bf16x2(f[6], f[7]));
    }
};
template <>
struct Raw8<float> {
    float4 x, y;
    __device__ __forceinline__ void load(const float* p)
    {
        x = reinterpret_cast<const float4*>(p)[0];
        y = reinterpret_cast<const float4*>(p)[1];
    }
    __device__ __forceinline__ void store(float* p) const
    {
        reinterpret_cast<float4*>(p)[0] = x;
        reinterpret_cast<float4*>(p)[1] = y;
    }
    __device__ __forceinline__ void get(float (&f)[8]) const
    {
        f[0] = x.x, f[1] = x.y, f[2] = x.z, f[3] = x.w;
        f[4] = y.x, f[5] = y.y, f[6] = y.z, f[7] = y.w;
    }
    __device__ __forceinline__ void set(const float (&f)[8])
    {
        x = make_float4(f[0], f[1], f[2], f[3]);
        y = make_float4(f[4], f[5], f[6], f[7]);
    }
};

// The rows of heads h, h + step, ... below h1 of one token: BATCH rows' loads
// are issued before the first is turned and stored.  x and out point at the
// token's row of head 0.
template <int BATCH, typename E>
__device__ __forceinline__ void rotate_heads(const RopeTable& t, bool turned, const float (&cs)[8],
                                             const float (&sn)[8], const E* x, int64_t x_sh,
                                             E* out, int64_t out_sh, int f0, int f1, int32_t h,
                                             int32_t h1, int32_t step)
{
    for (; h < h1; h += BATCH * step) {
        Raw8<E> r[BATCH][2];
#pragma unroll
        for (int k = 0; k < BATCH; ++k)
            if (h + k * step < h1) {
                r[k][0].load(x + (h + k * step) * x_sh + f0);
                r[k][1].load(x + (h + k * step) * x_sh + f1);
            }
#pragma unroll
        for (int k = 0; k < BATCH; ++k)
            if (h + k * step < h1) {
                if (turned) {
                    float a[8], b[8];
                    r[k][0].get(a);
                    r[k][1].get(b);
                    unit_rotate(t, cs, sn, a, b);
                    r[k][0].set(a);
                    r[k][1].set(b);
                }
                r[k][0].store(out + (h + k * step) * out_sh + f0);
                r[k][1].store(out + (h + k * step) * out_sh + f1);
            }
    }
}

// ---------------------------------------------------------------------------
// 8-bit cells (e4m3) with power-of-two scales
// ---------------------------------------------------------------------------
// The smallest power of two s >= 2^-100 with amax <= 448 s: 448 is 1.75 * 2^8,
// so the exponent goes up by one where amax's significand exceeds 1.75.
__device__ __forceinline__ float pow2_scale(float amax)
{
    const int e = (int)((__float_as_uint(amax) + 0x1fffffu) >> 23) - 127 - 8;
    return __uint_as_float((uint32_t)(max(e, -100) + 127) << 23);
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d)
{
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

// two codes (low, high byte) as fp16, exact
__device__ __forceinline__ uint32_t e4m3x2_half2(uint32_t codes)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
    return h;
}

__device__ __forceinline__ float2 e4m3x2_float2(uint32_t codes)
{
    const uint32_t h = e4m3x2_half2(codes);
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

}  // namespace dfa
