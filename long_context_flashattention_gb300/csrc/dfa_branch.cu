// dfa_branch.cu -- C ABI of the operators around branching sequences (include/dfa.h):
// trees of drafted tokens, kept rows, pools of shared pages.  Host code only.
#include "dfa_branch.h"
#include "dfa_checks.h"

using namespace dfa;
using namespace dfa::checks;

namespace {

dfa_status make_pool(PoolView* v, const dfa_page_pool* p, void* ws, const char* call)
{
    if (!p)
        return set_error(DFA_ERR_INVALID_ARG, "%s: pool is NULL", call);
    if (p->page != 16 && p->page != 32 && p->page != 64 && p->page != 128)
        return set_error(DFA_ERR_UNSUPPORTED, "%s: page must be 16, 32, 64 or 128", call);
    if (p->B < 1 || p->B > (1 << 20) || p->max_pages < 1 ||
        (int64_t)p->max_pages * p->page >= INT32_MAX / 2 ||
        (int64_t)p->max_pages * p->B >= INT32_MAX)
        return set_error(DFA_ERR_INVALID_ARG, "%s: need 1 <= B <= 2^20, max_pages >= 1, "
                         "max_pages * page < 2^30 and B * max_pages < 2^31 - 1", call);
    if (p->npages < 1 || p->npages >= INT32_MAX)
        return set_error(DFA_ERR_INVALID_ARG, "%s: npages must be in [1, 2^31 - 1)", call);
    if (!p->block_table || !p->held || !p->refs || !p->seq_lens)
        return set_error(DFA_ERR_INVALID_ARG, "%s: a pool pointer is NULL", call);
    if (((uintptr_t)p->status & 255u) != 0)
        return set_error(DFA_ERR_INVALID_ARG, "%s: status must be 256-byte aligned", call);
    v->table = p->block_table;
    v->held = p->held;
    v->refs = p->refs;
    v->seq_lens = p->seq_lens;
    v->npages = p->npages;
    v->B = p->B;
    v->max_pages = p->max_pages;
    v->page_log2 = p->page == 16 ? 4 : p->page == 32 ? 5 : p->page == 64 ? 6 : 7;
    v->status = (DevStatus*)(p->status ? p->status : ws);
    return DFA_OK;
}

// Workspace of the pool's calls: the status word, then fork's new rows of the table, or
// reserve's lists.
struct PoolWs {
    size_t rows, held, lens, fork_bytes;
    size_t offset, last, writers, free, reserve_bytes;
    PoolWs(int64_t B, int64_t max_pages, int64_t npages)
    {
        rows = kStatusBytes;
        held = rows + align256(B * max_pages * 4);
        lens = held + align256(B * 4);
        fork_bytes = lens + align256(B * 4);
        offset = kStatusBytes;
        last = offset + align256(B * 8);
        writers = last + align256(npages * 4);
        free = writers + align256(npages * 4);
        reserve_bytes = free + align256(npages * 4);
    }
};

// Workspace of dfa_decode_tree: status word, one record per block, two partial results
// (references and sum, O) per block, and what a block's two groups set apart of O.
struct TreeWs {
    size_t info, ndl, o, apart, bytes;
    explicit TreeWs(int d)
    {
        info = kStatusBytes;
        ndl = info + align256((size_t)kTreeMaxCtas * sizeof(int4));
        o = ndl + align256((size_t)2 * kTreeMaxCtas * kTreeRows * sizeof(float4));
        apart = o + align256((size_t)2 * kTreeMaxCtas * kTreeRows * d * 4);
        bytes = apart + (apart - o);
    }
};

dfa_status check_tree_tokens(int32_t T, const char* call)
{
    if (T < 1)
        return set_error(DFA_ERR_INVALID_ARG, "%s: T must be positive", call);
    if (T > kTreeMaxTokens)
        return set_error(DFA_ERR_UNSUPPORTED, "%s: at most %d tokens a tree", call,
                         kTreeMaxTokens);
    return DFA_OK;
}

}  // namespace

extern "C" {

dfa_status dfa_tree_plan(const dfa_paged_cache* cache, int32_t T, const int32_t* q_lens,
                         const int32_t* parents, uint32_t* mask, int32_t* positions, void* ws,
                         size_t ws_bytes, void* stream)
{
    TreePlanParams p;
    memset(&p, 0, sizeof p);
    dfa_status s = make_cache(&p.c, cache, ws, "dfa_tree_plan");
    if (s != DFA_OK)
        return s;
    if ((s = check_tree_tokens(T, "dfa_tree_plan")) != DFA_OK)
        return s;
    if (!parents || !mask || !positions)
        return set_error(DFA_ERR_INVALID_ARG, "dfa_tree_plan: parents, mask or positions is NULL");
    p.words = (T + 31) / 32;
    const size_t rows = (size_t)p.c.B * T * 4;
    if (spans_meet(parents, rows, mask, rows * p.words) ||
        spans_meet(parents, rows, positions, rows) ||
        spans_meet(positions, rows, mask, rows * p.words))
        return set_error(DFA_ERR_INVALID_ARG,
                         "dfa_tree_plan: parents, mask and positions overlap");
    if ((s = check_ws(ws, ws_bytes, kStatusBytes, "dfa_tree_plan")) != DFA_OK)
        return s;
    p.T = T;
    p.q_lens = q_lens;
    p.parents = parents;
    p.mask = mask;
    p.positions = positions;
    return launch_status(launch_tree_plan(p, (cudaStream_t)stream), "dfa_tree_plan");
}

size_t dfa_decode_tree_workspace_size(const dfa_attn_desc* desc, int32_t T)
{
    if (!desc || T < 1 || desc->Hkv < 1 || desc->Hq < 1 || desc->Hq % desc->Hkv != 0 ||
        (desc->d != 64 && desc->d != 128) || (int64_t)(desc->Hq / desc->Hkv) * T > 1024)
        return 0;
    return TreeWs(desc->d).bytes;
}

dfa_status dfa_decode_tree(const dfa_attn_desc* desc, const dfa_paged_cache* cache, int32_t T,
                           const int32_t* q_lens, const uint32_t* mask, const void* q,
                           const int64_t* q_strides, void* o, float* lse, void* ws,
                           size_t ws_bytes, void* stream)
{
    if (!desc)
        return set_error(DFA_ERR_INVALID_ARG, "dfa_decode_tree: desc is NULL");
    TreeParams p;
    memset(&p, 0, sizeof p);
    dfa_status s = make_cache(&p.c, cache, ws, "dfa_decode_tree");
    if (s != DFA_OK)
        return s;
    if (desc->B != p.c.B || desc->Hkv != p.c.Hkv || desc->d != p.c.d)
        return set_error(DFA_ERR_INVALID_ARG, "dfa_decode_tree: desc and cache differ in B, Hkv "
                         "or d");
    if (desc->Hq < 1 || desc->Hq % desc->Hkv != 0)
        return set_error(DFA_ERR_INVALID_ARG, "dfa_decode_tree: Hq (%d) must be a positive "
                         "multiple of Hkv (%d)", desc->Hq, desc->Hkv);
    const float scale_log2 = desc->scale * 1.4426950408889634f;
    if (!(scale_log2 > 0.f) || !std::isfinite(scale_log2))
        return set_error(DFA_ERR_INVALID_ARG, "dfa_decode_tree: scale must be positive and "
                         "finite, and so must scale * log2(e)");
    if (desc->o_fp32 != 0 && desc->o_fp32 != 1)
        return set_error(DFA_ERR_INVALID_ARG, "dfa_decode_tree: o_fp32 must be 0 or 1");
    if (desc->ndocs != 0)
        return set_error(DFA_ERR_UNSUPPORTED, "dfa_decode_tree takes no document bounds");
    if (T < 1)
        return set_error(DFA_ERR_INVALID_ARG, "dfa_decode_tree: T must be positive");
    const int G = desc->Hq / desc->Hkv;
    if ((int64_t)G * T > 1024)
        return set_error(DFA_ERR_UNSUPPORTED, "dfa_decode_tree: at most 1024 query rows per "
                         "key/value head (Hq/Hkv * T)");
    if ((s = make_rows(&p.q, q, q_strides, p.c.B, desc->Hq, T, p.c.d, 2, false,
                       "dfa_decode_tree: q")) != DFA_OK)
        return s;
    if (!mask || !o || !lse)
        return set_error(DFA_ERR_INVALID_ARG, "dfa_decode_tree: mask, o or lse is NULL");
    if (!aligned16(o))
        return set_error(DFA_ERR_UNSUPPORTED, "dfa_decode_tree: o must be 16-byte aligned");
    if ((s = check_ws(ws, ws_bytes, dfa_decode_tree_workspace_size(desc, T),
                      "dfa_decode_tree")) != DFA_OK)
        return s;
    // (blocks that read a sequence's queries and mask run beside one that writes its result)
    p.words = (T + 31) / 32;
    const size_t rows = (size_t)p.c.B * desc->Hq * T;
    const size_t q_bytes = span_bytes(p.q, p.c.B, desc->Hq, T, p.c.d, 2);
    const size_t mask_bytes = (size_t)p.c.B * T * p.words * 4;
    const size_t o_bytes = rows * p.c.d * (desc->o_fp32 ? 4 : 2);
    if (spans_meet(q, q_bytes, o, o_bytes) || spans_meet(q, q_bytes, lse, rows * 4) ||
        spans_meet(mask, mask_bytes, o, o_bytes) || spans_meet(mask, mask_bytes, lse, rows * 4) ||
        spans_meet(o, o_bytes, lse, rows * 4))
        return set_error(DFA_ERR_INVALID_ARG, "dfa_decode_tree: o and lse overlap one another or "
                         "q or mask");
    p.mask = mask;
    p.q_lens = q_lens;
    p.Hq = desc->Hq;
    p.G = G;
    p.T = T;
    p.inv_T = ((1u << 21) + T - 1) / T;
    p.o_fp32 = desc->o_fp32;
    p.scale_log2 = scale_log2;
    p.o = o;
    p.lse = lse;
    const TreeWs w(p.c.d);
    p.info = (int4*)((char*)ws + w.info);
    p.part_ndl = (float4*)((char*)ws + w.ndl);
    p.part_o = (float*)((char*)ws + w.o);
    p.apart = (float*)((char*)ws + w.apart);
    p.timeout_ns = kDefaultTimeoutNs;
    CUtensorMap tk, tv;
    if ((s = make_page_map(&tk, p.c, p.c.k, kTreeTile, "dfa_decode_tree: k")) != DFA_OK)
        return s;
    if ((s = make_page_map(&tv, p.c, p.c.v, kTreeTile, "dfa_decode_tree: v")) != DFA_OK)
        return s;
    return launch_status(launch_decode_tree(tk, tv, p, num_sms(), (cudaStream_t)stream),
                         "dfa_decode_tree");
}

dfa_status dfa_cache_compact(const dfa_paged_cache* cache, int32_t T, const int32_t* q_lens,
                             int32_t A, const int32_t* kept, const int32_t* kept_lens, void* ws,
                             size_t ws_bytes, void* stream)
{
    CompactParams p;
    memset(&p, 0, sizeof p);
    dfa_status s = make_cache(&p.c, cache, ws, "dfa_cache_compact");
    if (s != DFA_OK)
        return s;
    if (T < 1 || T >= (1 << 30) || A < 1 || A > T)
        return set_error(DFA_ERR_INVALID_ARG,
                         "dfa_cache_compact: need 1 <= A <= T and T < 2^30");
    if (!kept)
        return set_error(DFA_ERR_INVALID_ARG, "dfa_cache_compact: kept is NULL");
    if ((int64_t)2 * kCompactMaxParts * p.c.Hkv * p.c.B > kMaxBlocks)
        return set_error(DFA_ERR_UNSUPPORTED, "dfa_cache_compact: B * Hkv must be below 2^28");
    if ((s = check_ws(ws, ws_bytes, kStatusBytes, "dfa_cache_compact")) != DFA_OK)
        return s;
    p.q_lens = q_lens;
    p.kept = kept;
    p.kept_lens = kept_lens;
    p.T = T;
    p.A = A;
    return launch_status(launch_cache_compact(p, (cudaStream_t)stream), "dfa_cache_compact");
}

dfa_status dfa_cache_copy(const dfa_paged_cache* cache, const int32_t* jobs, int32_t max_jobs,
                          const int32_t* info, void* ws, size_t ws_bytes, void* stream)
{
    CopyParams p;
    memset(&p, 0, sizeof p);
    dfa_status s = make_cache(&p.c, cache, ws, "dfa_cache_copy");
    if (s != DFA_OK)
        return s;
    if (max_jobs < 1 || max_jobs >= (1 << 30))
        return set_error(DFA_ERR_INVALID_ARG, "dfa_cache_copy: max_jobs must be in [1, 2^30)");
    if (!jobs || !info)
        return set_error(DFA_ERR_INVALID_ARG, "dfa_cache_copy: jobs or info is NULL");
    if (((uintptr_t)jobs & 7u) != 0)
        return set_error(DFA_ERR_UNSUPPORTED, "dfa_cache_copy: jobs must be 8-byte aligned");
    if ((s = check_ws(ws, ws_bytes, kStatusBytes, "dfa_cache_copy")) != DFA_OK)
        return s;
    p.jobs = (const int2*)jobs;
    p.info = info;
    p.max_jobs = max_jobs;
    return launch_status(launch_cache_copy(p, num_sms(), (cudaStream_t)stream), "dfa_cache_copy");
}

size_t dfa_pages_workspace_size(const dfa_page_pool* pool)
{
    if (!pool || pool->B < 1 || pool->max_pages < 1 || pool->npages < 1)
        return 0;
    const PoolWs w(pool->B, pool->max_pages, pool->npages);
    return std::max(w.fork_bytes, w.reserve_bytes);
}

dfa_status dfa_pages_fork(const dfa_page_pool* pool, const int32_t* src, void* ws,
                          size_t ws_bytes, void* stream)
{
    ForkParams p;
    memset(&p, 0, sizeof p);
    dfa_status s = make_pool(&p.p, pool, ws, "dfa_pages_fork");
    if (s != DFA_OK)
        return s;
    if (!src)
        return set_error(DFA_ERR_INVALID_ARG, "dfa_pages_fork: src is NULL");
    const PoolWs w(p.p.B, p.p.max_pages, p.p.npages);
    if ((s = check_ws(ws, ws_bytes, w.fork_bytes, "dfa_pages_fork")) != DFA_OK)
        return s;
    p.src = src;
    p.rows = (int32_t*)((char*)ws + w.rows);
    p.held = (int32_t*)((char*)ws + w.held);
    p.lens = (int32_t*)((char*)ws + w.lens);
    return launch_status(launch_pages_fork(p, (cudaStream_t)stream), "dfa_pages_fork");
}

dfa_status dfa_pages_reserve(const dfa_page_pool* pool, int32_t T, const int32_t* new_lens,
                             int32_t* jobs, int32_t max_jobs, int32_t* info, void* ws,
                             size_t ws_bytes, void* stream)
{
    ReserveParams p;
    memset(&p, 0, sizeof p);
    dfa_status s = make_pool(&p.p, pool, ws, "dfa_pages_reserve");
    if (s != DFA_OK)
        return s;
    if (T < 0 || T >= (1 << 30))
        return set_error(DFA_ERR_INVALID_ARG, "dfa_pages_reserve: T must be in [0, 2^30)");
    if (max_jobs < 0 || max_jobs >= (1 << 30) || (max_jobs > 0 && !jobs))
        return set_error(DFA_ERR_INVALID_ARG, "dfa_pages_reserve: max_jobs must be in [0, 2^30), "
                         "and jobs not NULL unless it is 0");
    if (!info)
        return set_error(DFA_ERR_INVALID_ARG, "dfa_pages_reserve: info is NULL");
    if (((uintptr_t)jobs & 7u) != 0)
        return set_error(DFA_ERR_UNSUPPORTED, "dfa_pages_reserve: jobs must be 8-byte aligned");
    const PoolWs w(p.p.B, p.p.max_pages, p.p.npages);
    if ((s = check_ws(ws, ws_bytes, w.reserve_bytes, "dfa_pages_reserve")) != DFA_OK)
        return s;
    p.T = T;
    p.new_lens = new_lens;
    p.jobs = (int2*)jobs;
    p.max_jobs = max_jobs;
    p.info = info;
    p.offset = (int2*)((char*)ws + w.offset);
    p.last = (int32_t*)((char*)ws + w.last);
    p.writers = (int32_t*)((char*)ws + w.writers);
    p.free = (int32_t*)((char*)ws + w.free);
    return launch_status(launch_pages_reserve(p, (cudaStream_t)stream), "dfa_pages_reserve");
}

dfa_status dfa_pages_trim(const dfa_page_pool* pool, void* ws, size_t ws_bytes, void* stream)
{
    PoolView p;
    memset(&p, 0, sizeof p);
    dfa_status s = make_pool(&p, pool, ws, "dfa_pages_trim");
    if (s != DFA_OK)
        return s;
    if ((s = check_ws(ws, ws_bytes, kStatusBytes, "dfa_pages_trim")) != DFA_OK)
        return s;
    return launch_status(launch_pages_trim(p, (cudaStream_t)stream), "dfa_pages_trim");
}

}  // extern "C"
