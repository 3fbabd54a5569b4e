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
// of range is reported and makes the sequence empty.  (What kernels that are launched
// early read here, another may have written while they were there already: ordinary
// loads, not those for data that never changes during a kernel.  Loads from L2
// alone cost 0.4 us, since lengths are looked at several times.)
__device__ __forceinline__ void seq_rows(const CacheView& c, const int32_t* new_lens, int32_t T,
                                         int32_t b, int32_t& len, int32_t& n)
{
    len = c.seq_lens[b];
    n = new_lens ? new_lens[b] : T;
    if (len < 0 || len > (int64_t)c.max_pages * c.page) {
        cache_fault(c.status, kSiteSeqLen, b);
        len = n = 0;
    } else if (n < 0 || n > T || n > len) {
        cache_fault(c.status, kSiteNewLen, b);
        len = n = 0;
    }
}

// Table entry of rows [i*page, (i+1)*page) of sequence b, i < max_pages; and
// whether it is a page (if not, that is reported).  Apart, so that other loads
// can be on their way before the entry is looked at.
__device__ __forceinline__ int32_t page_entry(const CacheView& c, int32_t b, int32_t i)
{
    return c.table[(int64_t)b * c.max_pages + i];
}

__device__ __forceinline__ bool is_page(const CacheView& c, int32_t b, int32_t id)
{
    if (id >= 0 && id < c.npages)
        return true;
    cache_fault(c.status, kSitePage, b);
    return false;
}

// The page, or -1.
__device__ __forceinline__ int32_t page_of(const CacheView& c, int32_t b, int32_t i)
{
    const int32_t id = page_entry(c, b, i);
    return is_page(c, b, id) ? id : -1;
}

// ---------------------------------------------------------------------------
// rotation: a unit is V feature pairs (V features are 16 bytes), held by one lane
// as two runs of V features so that the lanes of a row load and store 16
// neighbouring bytes each.  Unit u of the U = rot_dim / 2V turned ones holds
// features Vu.. and rot_dim/2 + Vu..: in the half layout these are the two
// sides of pairs Vu.., in the interleaved one the pairs Vu/2.. and
// (rot_dim/2 + Vu)/2...  The other units split [rot_dim, d) likewise.
// ---------------------------------------------------------------------------
template <int V>
__device__ __forceinline__ bool unit_runs(const RopeTable& t, int d, int u, int& f0, int& f1)
{
    const int units = t.half / V;  // turned units
    const bool turned = u < units;
    f0 = turned ? V * u : 2 * t.half + V * (u - units);
    f1 = f0 + (turned ? t.half : d / 2 - t.half);
    return turned;
}

// Pair i (of V) of unit u.
template <int V>
__device__ __forceinline__ int unit_pair(const RopeTable& t, int u, int i)
{
    if (t.half_layout)
        return V * u + i;
    return V / 2 * u + i + (i < V / 2 ? 0 : t.half / 2 - V / 2);
}

// cos and sin (gain included) of a pair at a position.  The nearest whole quarter turn
// is taken out of the phase in integers, so that what is rounded to fp32, x in
// [-1/2, 1/2] quarter turns, is off by at most 2^-26 (2.4e-8 in the angle; the
// phase itself as fp32 would be by 9.4e-8).  Then the Taylor series of sin and cos(pi / 2 x),
// coefficients (pi / 2)^k / k!, which end at x^9 (2e-9) and x^10 (1e-10); the sine's
// first one in two terms.  In all they are off by at most 7.3e-8 (4 * 10^6 phases),
// sincospif from the phase by 1.2e-7.
__device__ __forceinline__ void pair_angle(uint64_t turn, float gain, int32_t pos, float sign,
                                           float& cs, float& sn)
{
    const uint64_t ph = (uint64_t)(int64_t)pos * turn;
    const uint32_t hi = (uint32_t)(ph >> 32);
    const float x = (float)(int32_t)__funnelshift_l((uint32_t)ph, hi, 2) * 0x1p-32f;
    const float x2 = x * x;
    float s = fmaf(1.6044118479e-4f, x2, -4.6817541353e-3f);
    s = fmaf(s, x2, 7.9692626246e-2f);
    s = fmaf(s, x2, -6.4596409751e-1f);
    s = fmaf(s, x2, -4.3711390063e-8f);  // pi / 2 less its fp32 value
    s = fmaf(x, 1.5707963268f, x * s);
    float c = fmaf(-2.5202042373e-5f, x2, 9.1926027484e-4f);
    c = fmaf(c, x2, -2.0863480763e-2f);
    c = fmaf(c, x2, 2.5366950790e-1f);
    c = fmaf(c, x2, -1.2337005501f);
    c = fmaf(c, x2, 1.f);
    const uint32_t quarter = ((hi >> 29) + 1) >> 1;
    const float u = quarter & 1 ? s : c, v = quarter & 1 ? c : s;
    cs = __uint_as_float(__float_as_uint(u) ^ ((quarter + 1) & 2) << 30) * gain;
    sn = __uint_as_float(__float_as_uint(v) ^ (quarter & 2) << 30) * (gain * sign);
}

// cos and sin of a unit's pairs where G * UNITS lanes are at one position, lane =
// (token * G + head) * UNITS + unit: the G lanes of a unit compute V / G pairs
// each and pass them around.
template <int V, int UNITS, int G>
struct SharedAngles {
    static constexpr int kOwn = V / G;
    uint64_t turn[kOwn];  // this lane's pairs
    float gain;

    // turns: the table's, in shared memory (the lanes read different entries)
    __device__ __forceinline__ SharedAngles(const RopeTable& t, const uint64_t* turns)
        : gain(t.gain)
    {
        const int lane = threadIdx.x & 31, u = lane & (UNITS - 1);
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
            const int pair = unit_pair<V>(t, u, lane / UNITS % G * kOwn + i);
            turn[i] = u < t.half / V ? turns[pair] : 0;
        }
    }
    __device__ __forceinline__ void at(int32_t pos, float sign, float (&cs)[V],
                                       float (&sn)[V]) const
    {
        const int lane = threadIdx.x & 31;
        const int first = lane & ~(G * UNITS - 1), u = lane & (UNITS - 1);
        float c[kOwn], s[kOwn];
#pragma unroll
        for (int i = 0; i < kOwn; ++i)
            pair_angle(turn[i], gain, pos, sign, c[i], s[i]);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            cs[i] = __shfl_sync(0xffffffffu, c[i % kOwn], first + (i / kOwn) * UNITS + u);
            sn[i] = __shfl_sync(0xffffffffu, s[i % kOwn], first + (i / kOwn) * UNITS + u);
        }
    }
};

// a, b: the unit's two runs
template <int V>
__device__ __forceinline__ void unit_rotate(const RopeTable& t, const float (&cs)[V],
                                            const float (&sn)[V], float (&a)[V], float (&b)[V])
{
    if (t.half_layout) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float x = a[i], y = b[i];
            a[i] = x * cs[i] - y * sn[i];
            b[i] = x * sn[i] + y * cs[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const float x = a[2 * i], y = a[2 * i + 1], z = b[2 * i], w = b[2 * i + 1];
            a[2 * i] = x * cs[i] - y * sn[i];
            a[2 * i + 1] = x * sn[i] + y * cs[i];
            b[2 * i] = z * cs[i + V / 2] - w * sn[i + V / 2];
            b[2 * i + 1] = z * sn[i + V / 2] + w * cs[i + V / 2];
        }
    }
}

// A run of 16 bytes: as it lies in memory, and as fp32.  (Plain loads: a call may
// work in place.)
template <typename E>
struct Run;
template <>
struct Run<__nv_bfloat16> {
    static constexpr int V = 8;
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
struct Run<float> {
    static constexpr int V = 4;
    float4 x;
    __device__ __forceinline__ void load(const float* p) { x = *reinterpret_cast<const float4*>(p); }
    __device__ __forceinline__ void store(float* p) const { *reinterpret_cast<float4*>(p) = x; }
    __device__ __forceinline__ void get(float (&f)[4]) const
    {
        f[0] = x.x, f[1] = x.y, f[2] = x.z, f[3] = x.w;
    }
    __device__ __forceinline__ void set(const float (&f)[4])
    {
        x = make_float4(f[0], f[1], f[2], f[3]);
    }
};

// Rows of tokens with few heads: lane = (token, head of G, unit), H <= G or, where
// the G heads take the whole warp, H <= 2 G.  A warp has BATCH rows a lane in
// flight, of as many tokens as that takes.  Rows: token(i) -> what is known
// of a token (pos; ok: there is such a row to move), from(token, h), to(token, h)
// (NULL: nowhere) and turns(h).
template <typename E, int D, int G, int BATCH, typename Rows>
__device__ __forceinline__ void few_heads(const RopeTable& t, const uint64_t* turns,
                                          const Rows& rows, int32_t H, uint32_t tokens, float sign,
                                          uint32_t warp, uint32_t warps)
{
    constexpr int V = Run<E>::V, UNITS = D / (2 * V), kTokens = 32 / UNITS / G;
    const int lane = threadIdx.x & 31, u = lane & (UNITS - 1);
    const int32_t h = lane / UNITS % G;
    const uint32_t mine = lane / UNITS / G;  // token of the kTokens at a time
    const int twice = H > G ? 1 : 0;         // two heads of a token a lane
    const uint32_t each = (BATCH >> twice) * kTokens;
    int f0, f1;
    const bool turned = unit_runs<V>(t, D, u, f0, f1);
    const SharedAngles<V, UNITS, G> angles(t, turns);
    for (uint32_t first = warp * each; first < tokens; first += warps * each) {
        typename Rows::Token tok[BATCH];
        Run<E> r[BATCH][2];
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const uint32_t i = first + (k >> twice) * kTokens + mine;
            const int32_t hk = h + (k & twice) * G;
            tok[k] = rows.token(min(i, tokens - 1));
            tok[k].ok = tok[k].ok && i < tokens && hk < H;
            if (tok[k].ok) {
                const E* x = rows.from(tok[k], hk);
                r[k][0].load(x + f0);
                r[k][1].load(x + f1);
            }
        }
        float cs[V], sn[V];
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const int32_t hk = h + (k & twice) * G;
            if (!(k & twice))
                angles.at(tok[k].pos, sign, cs, sn);
            E* to = tok[k].ok ? rows.to(tok[k], hk) : nullptr;
            if (!to)
                continue;
            if (turned && rows.turns(hk)) {
                float a[V], c[V];
                r[k][0].get(a);
                r[k][1].get(c);
                unit_rotate<V>(t, cs, sn, a, c);
                r[k][0].set(a);
                r[k][1].set(c);
            }
            r[k][0].store(to + f0);
            r[k][1].store(to + f1);
        }
    }
}

// Heads a step of `step` that few_heads takes H of: the power of two.
inline int few_heads_group(int H, int step)
{
    int g = 1;
    while (g < H && g < step)
        g *= 2;
    return g;
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
