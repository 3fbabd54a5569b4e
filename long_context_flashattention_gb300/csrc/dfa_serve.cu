// dfa_serve.cu -- C ABI of rotary positions and of the paged key/value cache
// (include/dfa.h): argument checks, frequency tables, launches.  Host code only.
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
}

using namespace dfa;

namespace {

constexpr size_t kStatusBytes = 256;
constexpr int64_t kMaxBlocks = INT32_MAX;
constexpr uint64_t kDefaultTimeoutNs = 4000000000ull;  // 4 s per wait

int num_sms()
{
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return 1;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 1;
    return n > 0 ? n : 1;
}

dfa_status launch_status(cudaError_t e, const char* call)
{
    if (e == cudaSuccess)
        return DFA_OK;
    return set_error(DFA_ERR_CUDA, "%s: %s", call, cudaGetErrorString(e));
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

dfa_status check_ws(void* ws, size_t have, size_t need, const char* call)
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
dfa_status make_rows(Rows* r, const void* p, const int64_t* strides, int64_t B, int64_t H,
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
size_t span_bytes(const Rows& r, int64_t B, int64_t H, int64_t L, int d, int elem_bytes)
{
    return (size_t)((B - 1) * r.sb + (H - 1) * r.sh + (L - 1) * r.sl + d) * elem_bytes;
}

bool spans_meet(const void* a, size_t a_bytes, const void* b, size_t b_bytes)
{
    return (const char*)a < (const char*)b + b_bytes && (const char*)b < (const char*)a + a_bytes;
}

// Two tensors of one shape: the same one (in place), or apart.
dfa_status check_apart(const Rows& x, const Rows& out, int64_t B, int64_t H, int64_t L, int d,
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

dfa_status make_table(RopeTable* t, const dfa_rope_spec* s, int d)
{
    memset(t, 0, sizeof *t);
    if (!s)
        return DFA_OK;  // no rotation: every unit passes through
    if (s->layout != DFA_ROPE_INTERLEAVED && s->layout != DFA_ROPE_HALF)
        return set_error(DFA_ERR_INVALID_ARG, "rope: unknown layout %d", s->layout);
    if (s->rot_dim < 2 || s->rot_dim > d || s->rot_dim % 2 != 0)
        return set_error(DFA_ERR_INVALID_ARG, "rope: rot_dim must be even, in [2, d]");
    if (s->rot_dim % 16 != 0)
        return set_error(DFA_ERR_UNSUPPORTED, "rope: rot_dim must be a multiple of 16");
    if (!(s->theta_base > 1.0) || !std::isfinite(s->theta_base))
        return set_error(DFA_ERR_INVALID_ARG, "rope: theta_base must be finite and > 1");
    const double gain = s->gain == 0.0 ? 1.0 : s->gain;
    if (!((float)gain > 0.f) || !std::isfinite((float)gain))
        return set_error(DFA_ERR_INVALID_ARG, "rope: gain must be positive and finite in fp32");
    if (s->scaling < DFA_ROPE_PLAIN || s->scaling > DFA_ROPE_BANDS)
        return set_error(DFA_ERR_INVALID_ARG, "rope: unknown scaling %d", s->scaling);
    if (s->scaling != DFA_ROPE_PLAIN && (!(s->factor > 0.0) || !std::isfinite(s->factor)))
        return set_error(DFA_ERR_INVALID_ARG, "rope: factor must be positive and finite");
    if (s->scaling == DFA_ROPE_BANDS &&
        (!(s->orig_len > 0.0) || !std::isfinite(s->orig_len) || !(s->low >= 0.0) ||
         !(s->high > s->low) || !std::isfinite(s->high)))
        return set_error(DFA_ERR_INVALID_ARG,
                         "rope: bands need orig_len > 0 and 0 <= low < high, all finite");
    // The frequencies take longer than a launch, and calls repeat their spec.
    thread_local struct {
        dfa_rope_spec spec;
        RopeTable table;
        bool valid = false;
    } last;
    if (last.valid && memcmp(&last.spec, s, sizeof *s) == 0) {
        *t = last.table;
        return DFA_OK;
    }
    constexpr double kTwoPi = 6.283185307179586;
    t->gain = (float)gain;
    t->half_layout = s->layout == DFA_ROPE_HALF;
    t->half = s->rot_dim / 2;
    for (int i = 0; i < t->half; ++i) {
        double f = std::pow(s->theta_base, -2.0 * i / s->rot_dim);
        if (s->scaling == DFA_ROPE_LINEAR) {
            f /= s->factor;
        } else if (s->scaling == DFA_ROPE_BANDS) {
            const double turns = s->orig_len * f / kTwoPi;
            const double u =
                std::min(1.0, std::max(0.0, (turns - s->low) / (s->high - s->low)));
            f = (1.0 - u) * f / s->factor + u * f;
        }
        if (!std::isfinite(f))
            return set_error(DFA_ERR_INVALID_ARG, "rope: a frequency is not finite");
        double turn = f / kTwoPi;  // whole turns of an integer position drop out
        turn -= std::floor(turn);
        t->turn[i] = (uint64_t)std::ldexp(turn, 64);  // turn < 1: below 2^64
    }
    last.spec = *s;
    last.table = *t;
    last.valid = true;
    return DFA_OK;
}

dfa_status make_cache(CacheView* v, const dfa_paged_cache* c, void* ws, const char* call)
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
// features by up to 64 rows, swizzled by the box's width.
dfa_status make_page_map(CUtensorMap* out, const CacheView& c, const void* ptr, const char* name)
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
        return set_error(DFA_ERR_CUDA, "dfa_decode_paged: cuTensorMapEncodeTiled unavailable");
    const int es = c.e4m3 ? 1 : 2;
    const int box_bytes = std::min(128, c.d * es);
    cuuint64_t dims[4] = {(cuuint64_t)c.d, (cuuint64_t)c.page, (cuuint64_t)c.Hkv,
                          (cuuint64_t)c.npages};
    cuuint64_t strides[3] = {(cuuint64_t)c.d * es, (cuuint64_t)c.page * c.d * es,
                             (cuuint64_t)c.page_stride * es};
    cuuint32_t box[4] = {(cuuint32_t)(box_bytes / es),
                         (cuuint32_t)std::min(c.page, kPagedTile), 1, 1};
    cuuint32_t step[4] = {1, 1, 1, 1};
    const CUresult r =
        fn(out, c.e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
           const_cast<void*>(ptr), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
           box_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return set_error(DFA_ERR_CUDA, "dfa_decode_paged: tensor map for %s failed (CUresult %d)",
                         name, (int)r);
    return DFA_OK;
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Query rows of a block: 8, or 16 where a key/value head has more.
int paged_rows(int64_t rows_per_head)
{
    return rows_per_head <= kPagedRows ? kPagedRows : kPagedMaxRows;
}

// Workspace of dfa_decode_paged: status word, one record per block, two partial
// results (references and sum, O) per block.
struct PagedWs {
    size_t info, ndl, o, bytes;
    PagedWs(int rows, int d)
    {
        info = kStatusBytes;
        ndl = info + align256((size_t)kPagedMaxCtas * sizeof(int4));
        o = ndl + align256((size_t)2 * kPagedMaxCtas * rows * sizeof(float4));
        bytes = o + align256((size_t)2 * kPagedMaxCtas * rows * d * 4);
    }
};

}  // namespace

extern "C" {

dfa_status dfa_rope(const dfa_rope_spec* spec, int32_t B, int32_t H, int64_t L, int32_t d,
                    int32_t fp32, const void* x, const int64_t* x_strides, void* out,
                    const int64_t* out_strides, const dfa_pos_map* map,
                    const int32_t* positions, int32_t inverse, void* stream)
{
    if (!spec)
        return set_error(DFA_ERR_INVALID_ARG, "dfa_rope: spec is NULL");
    if (B < 1 || H < 1 || L < 0)
        return set_error(DFA_ERR_INVALID_ARG, "dfa_rope: need B, H >= 1 and L >= 0");
    if (B > (1 << 20) || H > (1 << 20) || L >= (1 << 30) ||
        (int64_t)B * H >= kMaxBlocks || (int64_t)B * H * L >= kMaxBlocks)
        return set_error(DFA_ERR_UNSUPPORTED, "dfa_rope: B and H up to 2^20, L below 2^30, "
                         "B * H * L below 2^31");
    if (d != 64 && d != 128)
        return set_error(DFA_ERR_UNSUPPORTED, "dfa_rope: head dimension %d not supported "
                         "(64 or 128)", d);
    if ((fp32 != 0 && fp32 != 1) || (inverse != 0 && inverse != 1))
        return set_error(DFA_ERR_INVALID_ARG, "dfa_rope: fp32 and inverse must be 0 or 1");
    RopeRowsParams p;
    memset(&p, 0, sizeof p);
    dfa_status s = make_table(&p.t, spec, d);
    if (s != DFA_OK)
        return s;
    const int eb = fp32 ? 4 : 2;
    p.map.blk = p.map.blk_stride = 1;
    p.map.len0 = (int32_t)L;
    if (map && !positions) {
        const int64_t l1 = map->nseg == 2 ? map->len[1] : 0;
        if ((map->nseg != 1 && map->nseg != 2) || map->len[0] < 0 || l1 < 0 ||
            map->len[0] + l1 != L)
            return set_error(DFA_ERR_INVALID_ARG, "dfa_rope: map must have 1 or 2 segments of "
                             "%lld rows in all", (long long)L);
        if (map->blk < 1 || map->blk_stride < map->blk || map->blk_stride > INT32_MAX)
            return set_error(DFA_ERR_UNSUPPORTED, "dfa_rope: map needs 1 <= blk <= blk_stride");
        for (int i = 0; i < map->nseg; ++i) {
            const int64_t len = map->len[i];
            if (len == 0)
                continue;
            // quotient first: the product could pass 64 bits for wild strides
            const int64_t steps = (len - 1) / map->blk;
            if (map->base[i] < 0 || map->base[i] >= INT32_MAX ||
                map->base[i] + steps * map->blk_stride + (len - 1) % map->blk >= INT32_MAX)
                return set_error(DFA_ERR_UNSUPPORTED,
                                 "dfa_rope: positions of map must lie in [0, 2^31)");
        }
        p.map.len0 = (int32_t)map->len[0];
        p.map.len1 = (int32_t)l1;
        p.map.base0 = map->len[0] ? (int32_t)map->base[0] : 0;
        p.map.base1 = l1 ? (int32_t)map->base[1] : 0;
        p.map.blk = (int32_t)std::min<int64_t>(map->blk, INT32_MAX);
        p.map.blk_stride = (int32_t)map->blk_stride;
    }
    if (L == 0)
        return DFA_OK;
    if ((s = make_rows(&p.x, x, x_strides, B, H, L, d, eb, false, "dfa_rope: x")) != DFA_OK)
        return s;
    if ((s = make_rows(&p.out, out, out_strides, B, H, L, d, eb, true, "dfa_rope: out")) != DFA_OK)
        return s;
    if ((s = check_apart(p.x, p.out, B, H, L, d, eb, "dfa_rope: x and out")) != DFA_OK)
        return s;
    p.B = B;
    p.H = H;
    p.L = L;
    p.d = d;
    p.inverse = inverse;
    p.positions = positions;
    return launch_status(launch_rope_rows(p, fp32, num_sms(), (cudaStream_t)stream), "dfa_rope");
}

dfa_status dfa_cache_append(const dfa_paged_cache* cache, const dfa_rope_spec* rope, int32_t T,
                            const int32_t* new_lens, const void* k, const int64_t* k_strides,
                            const void* v, const int64_t* v_strides, int32_t Hq, const void* q,
                            const int64_t* q_strides, void* q_out, const int64_t* q_out_strides,
                            void* ws, size_t ws_bytes, void* stream)
{
    AppendParams p;
    memset(&p, 0, sizeof p);
    dfa_status s = make_cache(&p.c, cache, ws, "dfa_cache_append");
    if (s != DFA_OK)
        return s;
    const int32_t B = p.c.B, Hkv = p.c.Hkv, d = p.c.d, page = p.c.page;
    if (T < 1 || T >= (1 << 30))
        return set_error(DFA_ERR_INVALID_ARG, "dfa_cache_append: T must be in [1, 2^30)");
    if ((s = make_table(&p.t, rope, d)) != DFA_OK)
        return s;
    if ((s = make_rows(&p.k, k, k_strides, B, Hkv, T, d, 2, false, "dfa_cache_append: k")) !=
        DFA_OK)
        return s;
    if ((s = make_rows(&p.v, v, v_strides, B, Hkv, T, d, 2, false, "dfa_cache_append: v")) !=
        DFA_OK)
        return s;
    if (q) {
        if (!rope)
            return set_error(DFA_ERR_INVALID_ARG, "dfa_cache_append: queries without a rotation");
        if (Hq < 1 || Hq > (1 << 20))
            return set_error(DFA_ERR_INVALID_ARG, "dfa_cache_append: Hq must be in [1, 2^20]");
        if ((s = make_rows(&p.q, q, q_strides, B, Hq, T, d, 2, false, "dfa_cache_append: q")) !=
            DFA_OK)
            return s;
        if ((s = make_rows(&p.q_out, q_out, q_out_strides, B, Hq, T, d, 2, true,
                           "dfa_cache_append: q_out")) != DFA_OK)
            return s;
        if ((s = check_apart(p.q, p.q_out, B, Hq, T, d, 2, "dfa_cache_append: q and q_out")) !=
            DFA_OK)
            return s;
        p.Hq = Hq;
    }
    if ((s = check_ws(ws, ws_bytes, kStatusBytes, "dfa_cache_append")) != DFA_OK)
        return s;
    p.new_lens = new_lens;
    p.T = T;
    // T rows touch at most this many pages, and never more than a sequence has
    p.pages = std::min(p.c.max_pages, (int32_t)(((int64_t)T + page - 2) / page + 1));
    if ((int64_t)B * T * (p.Hq + 2 * Hkv) >= kMaxBlocks)
        return set_error(DFA_ERR_UNSUPPORTED, "dfa_cache_append: B * T * heads above 2^31");
    return launch_status(launch_cache_append(p, num_sms(), (cudaStream_t)stream),
                         "dfa_cache_append");
}

dfa_status dfa_cache_gather(const dfa_paged_cache* cache, int64_t pos0, int64_t L, void* k_out,
                            void* v_out, void* ws, size_t ws_bytes, void* stream)
{
    GatherParams p;
    memset(&p, 0, sizeof p);
    dfa_status s = make_cache(&p.c, cache, ws, "dfa_cache_gather");
    if (s != DFA_OK)
        return s;
    if (pos0 < 0 || L < 0 || pos0 >= (1 << 30) || L >= (1 << 30))
        return set_error(DFA_ERR_INVALID_ARG, "dfa_cache_gather: pos0 and L must be in [0, 2^30)");
    if (!aligned16(k_out) || !aligned16(v_out))
        return set_error(DFA_ERR_UNSUPPORTED, "dfa_cache_gather: outputs must be 16-byte aligned");
    if ((s = check_ws(ws, ws_bytes, kStatusBytes, "dfa_cache_gather")) != DFA_OK)
        return s;
    p.pos0 = pos0;
    p.L = L;
    p.k_out = k_out;
    p.v_out = v_out;
    const int64_t rows = (int64_t)p.c.max_pages * p.c.page;
    const int64_t end = std::min(pos0 + L, rows);
    if (pos0 >= end || (!k_out && !v_out))
        return DFA_OK;  // no such rows
    const size_t out_bytes = (size_t)p.c.B * p.c.Hkv * L * p.c.d * 2;
    if (k_out && v_out && spans_meet(k_out, out_bytes, v_out, out_bytes))
        return set_error(DFA_ERR_INVALID_ARG, "dfa_cache_gather: k_out and v_out overlap");
    p.page0 = (int32_t)(pos0 / p.c.page);
    p.pages = (int32_t)((end - 1) / p.c.page) - p.page0 + 1;
    if ((int64_t)p.pages * p.c.Hkv * p.c.B > kMaxBlocks)
        return set_error(DFA_ERR_UNSUPPORTED, "dfa_cache_gather: too many rows for one call");
    return launch_status(launch_cache_gather(p, (cudaStream_t)stream), "dfa_cache_gather");
}

size_t dfa_decode_paged_workspace_size(const dfa_attn_desc* desc, int32_t T)
{
    if (!desc || T < 1 || desc->Hkv < 1 || desc->Hq < 1 || desc->Hq % desc->Hkv != 0 ||
        (desc->d != 64 && desc->d != 128) || (int64_t)(desc->Hq / desc->Hkv) * T > 1024)
        return 0;
    return PagedWs(paged_rows((int64_t)(desc->Hq / desc->Hkv) * T), desc->d).bytes;
}

dfa_status dfa_decode_paged(const dfa_attn_desc* desc, const dfa_paged_cache* cache, int32_t T,
                            const int32_t* q_lens, const void* q, const int64_t* q_strides,
                            void* o, float* lse, void* ws, size_t ws_bytes, void* stream)
{
    if (!desc)
        return set_error(DFA_ERR_INVALID_ARG, "dfa_decode_paged: desc is NULL");
    PagedParams p;
    memset(&p, 0, sizeof p);
    dfa_status s = make_cache(&p.c, cache, ws, "dfa_decode_paged");
    if (s != DFA_OK)
        return s;
    if (desc->B != p.c.B || desc->Hkv != p.c.Hkv || desc->d != p.c.d)
        return set_error(DFA_ERR_INVALID_ARG, "dfa_decode_paged: desc and cache differ in B, Hkv "
                         "or d");
    if (desc->Hq < 1 || desc->Hq % desc->Hkv != 0)
        return set_error(DFA_ERR_INVALID_ARG, "dfa_decode_paged: Hq (%d) must be a positive "
                         "multiple of Hkv (%d)", desc->Hq, desc->Hkv);
    const float scale_log2 = desc->scale * 1.4426950408889634f;
    if (!(scale_log2 > 0.f) || !std::isfinite(scale_log2))
        return set_error(DFA_ERR_INVALID_ARG, "dfa_decode_paged: scale must be positive and "
                         "finite, and so must scale * log2(e)");
    if (desc->causal != 0 && desc->causal != 1)
        return set_error(DFA_ERR_INVALID_ARG, "dfa_decode_paged: causal must be 0 or 1");
    if (desc->o_fp32 != 0 && desc->o_fp32 != 1)
        return set_error(DFA_ERR_INVALID_ARG, "dfa_decode_paged: o_fp32 must be 0 or 1");
    if (desc->ndocs != 0)
        return set_error(DFA_ERR_UNSUPPORTED, "dfa_decode_paged takes no document bounds");
    if (T < 1)
        return set_error(DFA_ERR_INVALID_ARG, "dfa_decode_paged: T must be positive");
    const int G = desc->Hq / desc->Hkv;
    if ((int64_t)G * T > 1024)
        return set_error(DFA_ERR_UNSUPPORTED, "dfa_decode_paged: at most 1024 query rows per "
                         "key/value head (Hq/Hkv * T)");
    if ((s = make_rows(&p.q, q, q_strides, p.c.B, desc->Hq, T, p.c.d, 2, false,
                       "dfa_decode_paged: q")) != DFA_OK)
        return s;
    if (!o || !lse)
        return set_error(DFA_ERR_INVALID_ARG, "dfa_decode_paged: o or lse is NULL");
    if (!aligned16(o))
        return set_error(DFA_ERR_UNSUPPORTED, "dfa_decode_paged: o must be 16-byte aligned");
    const size_t need = dfa_decode_paged_workspace_size(desc, T);
    if ((s = check_ws(ws, ws_bytes, need, "dfa_decode_paged")) != DFA_OK)
        return s;
    // (blocks that read a sequence's queries run beside one that writes its result)
    if (spans_meet(q, span_bytes(p.q, p.c.B, desc->Hq, T, p.c.d, 2), o,
                   (size_t)p.c.B * desc->Hq * T * p.c.d * (desc->o_fp32 ? 4 : 2)))
        return set_error(DFA_ERR_INVALID_ARG, "dfa_decode_paged: q and o overlap");
    p.q_lens = q_lens;
    p.Hq = desc->Hq;
    p.G = G;
    p.T = T;
    p.inv_T = ((1u << 21) + T - 1) / T;
    p.causal = desc->causal;
    p.o_fp32 = desc->o_fp32;
    p.scale_log2 = scale_log2;
    p.o = o;
    p.lse = lse;
    const int rows = paged_rows((int64_t)G * T);
    const PagedWs w(rows, p.c.d);
    p.row_groups = (G * T + rows - 1) / rows;
    p.info = (int4*)((char*)ws + w.info);
    p.part_ndl = (float4*)((char*)ws + w.ndl);
    p.part_o = (float*)((char*)ws + w.o);
    p.timeout_ns = kDefaultTimeoutNs;
    CUtensorMap tk, tv;
    if ((s = make_page_map(&tk, p.c, p.c.k, "k")) != DFA_OK)
        return s;
    if ((s = make_page_map(&tv, p.c, p.c.v, "v")) != DFA_OK)
        return s;
    return launch_status(launch_decode_paged(tk, tv, p, num_sms(), (cudaStream_t)stream),
                         "dfa_decode_paged");
}

}  // extern "C"
