// dfa_checks.h -- host-side checks shared by the entries of the serving operators:
// row tensors, paged caches, workspaces, tensor maps of pages.
#pragma once

#include <algorithm>
#include <cmath>
#include <cstring>

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include "../../include/dfa.h"
#include "dfa_serve.h"

namespace dfa {

dfa_status set_error(dfa_status s, const char* fmt, ...);

namespace checks {

constexpr size_t kStatusBytes = 256;
constexpr int64_t kMaxBlocks = INT32_MAX;
constexpr uint64_t kDefaultTimeoutNs = 4000000000ull;  // 4 s per wait

inline int num_sms()
{
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return 1;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 1;
    return n > 0 ? n : 1;
}

inline dfa_status launch_status(cudaError_t e, const char* call)
{
    if (e == cudaSuccess)
        return DFA_OK;
    return set_error(DFA_ERR_CUDA, "%s: %s", call, cudaGetErrorString(e));
}

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

inline dfa_status check_ws(void* ws, size_t have, size_t need, const char* call)
{
    if (!ws)
        return set_error(DFA_ERR_WORKSPACE, "%s: workspace is NULL", call);
    if (((uintptr_t)ws & 255u) != 0)
        return set_error(DFA_ERR_WORKSPACE, "%s: workspace must be 256-byte aligned", call);
    if (have < need)
        return set_error(DFA_ERR_WORKSPACE, "%s: workspace too small: %zu < %zu", call, have, need);
    return DFA_OK;
}

// A row tensor [B, H, L, d] of elem_bytes elements.  out: rows must be apart.
inline dfa_status make_rows(Rows* r, const void* p, const int64_t* strides, int64_t B, int64_t H,
                     int64_t L, int d, int elem_bytes, bool out, const char* name)
{
    if (!p)
        return set_error(DFA_ERR_INVALID_ARG, "%s is NULL", name);
    r->p = const_cast<void*>(p);
    r->sb = strides ? strides[0] : H * L * d;
    r->sh = strides ? strides[1] : L * d;
    r->sl = strides ? strides[2] : d;
    struct Dim {
        int64_t n, s;
    } dims[3] = {{B, r->sb}, {H, r->sh}, {L, r->sl}};
    for (const Dim& x : dims) {
        if (x.n <= 1)
            continue;
        if (x.s < 0 || x.s > (INT64_C(1) << 40))
            return set_error(DFA_ERR_INVALID_ARG, "%s: strides must lie in [0, 2^40]", name);
        if (x.s * elem_bytes % 16 != 0)
            return set_error(DFA_ERR_UNSUPPORTED, "%s: strides must be multiples of 16 bytes",
                             name);
    }
    if (!aligned16(p))
        return set_error(DFA_ERR_UNSUPPORTED, "%s must be 16-byte aligned", name);
    if (out) {
        std::sort(dims, dims + 3, [](const Dim& x, const Dim& y) { return x.s < y.s; });
        int64_t extent = d;  // elements spanned by the dimensions so far
        for (const Dim& x : dims) {
            if (x.n <= 1)
                continue;
            if (x.s < extent)
                return set_error(DFA_ERR_INVALID_ARG, "%s: rows overlap one another", name);
            extent += (x.n - 1) * x.s;
        }
    }
    return DFA_OK;
}

// Bytes from a tensor's first row to the end of its last.
inline size_t span_bytes(const Rows& r, int64_t B, int64_t H, int64_t L, int d, int elem_bytes)
{
    return (size_t)((B - 1) * r.sb + (H - 1) * r.sh + (L - 1) * r.sl + d) * elem_bytes;
}

inline bool spans_meet(const void* a, size_t a_bytes, const void* b, size_t b_bytes)
{
    return (const char*)a < (const char*)b + b_bytes && (const char*)b < (const char*)a + a_bytes;
}

// Two tensors of one shape: the same one (in place), or apart.
inline dfa_status check_apart(const Rows& x, const Rows& out, int64_t B, int64_t H, int64_t L, int d,
                       int elem_bytes, const char* names)
{
    if (x.p == out.p && (B <= 1 || x.sb == out.sb) && (H <= 1 || x.sh == out.sh) &&
        (L <= 1 || x.sl == out.sl))
        return DFA_OK;
    if (spans_meet(x.p, span_bytes(x, B, H, L, d, elem_bytes), out.p,
                   span_bytes(out, B, H, L, d, elem_bytes)))
        return set_error(DFA_ERR_INVALID_ARG, "%s overlap without being the same tensor", names);
    return DFA_OK;
}

inline dfa_status make_cache(CacheView* v, const dfa_paged_cache* c, void* ws, const char* call)
{
    if (!c)
        return set_error(DFA_ERR_INVALID_ARG, "%s: cache is NULL", call);
    if (c->dtype != DFA_CACHE_BF16 && c->dtype != DFA_CACHE_E4M3)
        return set_error(DFA_ERR_INVALID_ARG, "%s: unknown cache dtype %d", call, c->dtype);
    if (c->d != 64 && c->d != 128)
        return set_error(DFA_ERR_UNSUPPORTED, "%s: head dimension %d not supported (64 or 128)",
                         call, c->d);
    if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128)
        return set_error(DFA_ERR_UNSUPPORTED, "%s: page must be 16, 32, 64 or 128", call);
    if (c->Hkv < 1 || c->Hkv > 65535 || c->B < 1 || c->B > (1 << 20) || c->max_pages < 1 ||
        (int64_t)c->max_pages * c->page >= INT32_MAX / 2)
        return set_error(DFA_ERR_INVALID_ARG, "%s: need 1 <= Hkv < 2^16, 1 <= B <= 2^20, "
                         "max_pages >= 1 and max_pages * page < 2^30", call);
    if (c->npages < 1 || c->npages >= INT32_MAX)
        return set_error(DFA_ERR_INVALID_ARG, "%s: npages must be in [1, 2^31 - 1)", call);
    const bool e4m3 = c->dtype == DFA_CACHE_E4M3;
    const int64_t whole = (int64_t)c->Hkv * c->page * c->d;
    const int64_t stride = c->page_stride ? c->page_stride : whole;
    if (stride < whole || stride > (INT64_C(1) << 36))
        return set_error(DFA_ERR_INVALID_ARG, "%s: page_stride must be in [Hkv*page*d, 2^36]",
                         call);
    if (stride * (e4m3 ? 1 : 2) % 16 != 0)
        return set_error(DFA_ERR_UNSUPPORTED, "%s: page_stride must be a multiple of 16 bytes",
                         call);
    if (!c->k || !c->v || !c->block_table || !c->seq_lens || (e4m3 && (!c->k_scale || !c->v_scale)))
        return set_error(DFA_ERR_INVALID_ARG, "%s: a cache pointer is NULL", call);
    if (!aligned16(c->k) || !aligned16(c->v))
        return set_error(DFA_ERR_UNSUPPORTED, "%s: k and v must be 16-byte aligned", call);
    if (((uintptr_t)c->status & 255u) != 0)
        return set_error(DFA_ERR_INVALID_ARG, "%s: status must be 256-byte aligned", call);
    v->k = c->k;
    v->v = c->v;
    v->k_scale = e4m3 ? c->k_scale : nullptr;
    v->v_scale = e4m3 ? c->v_scale : nullptr;
    v->table = c->block_table;
    v->seq_lens = c->seq_lens;
    v->npages = c->npages;
    v->page_stride = stride;
    v->B = c->B;
    v->Hkv = c->Hkv;
    v->d = c->d;
    v->page = c->page;
    v->page_log2 = c->page == 16 ? 4 : c->page == 32 ? 5 : c->page == 64 ? 6 : 7;
    v->max_pages = c->max_pages;
    v->e4m3 = e4m3;
    v->status = (DevStatus*)(c->status ? c->status : ws);
    return DFA_OK;
}

// Pages as a tensor map [npages][Hkv][page][d] with boxes of up to 128 bytes of
// features by up to box_rows rows, swizzled by the box's width.
inline dfa_status make_page_map(CUtensorMap* out, const CacheView& c, const void* ptr, int box_rows,
                                const char* name)
{
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return (PFN_cuTensorMapEncodeTiled_v12000)p;
    }();
    if (!fn)
        return set_error(DFA_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
    const int es = c.e4m3 ? 1 : 2;
    const int box_bytes = std::min(128, c.d * es);
    cuuint64_t dims[4] = {(cuuint64_t)c.d, (cuuint64_t)c.page, (cuuint64_t)c.Hkv,
                          (cuuint64_t)c.npages};
    cuuint64_t strides[3] = {(cuuint64_t)c.d * es, (cuuint64_t)c.page * c.d * es,
                             (cuuint64_t)c.page_stride * es};
    cuuint32_t box[4] = {(cuuint32_t)(box_bytes / es),
                         (cuuint32_t)std::min(c.page, box_rows), 1, 1};
    cuuint32_t step[4] = {1, 1, 1, 1};
    const CUresult r =
        fn(out, c.e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
           const_cast<void*>(ptr), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
           box_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return set_error(DFA_ERR_CUDA, "tensor map for %s failed (CUresult %d)",
                         name, (int)r);
    return DFA_OK;
}

inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace checks
}  // namespace dfa
