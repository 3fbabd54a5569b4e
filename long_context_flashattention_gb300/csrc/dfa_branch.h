// dfa_branch.h -- plain-data structures of the operators around branching sequences:
// trees of drafted tokens over a paged cache, kept rows, and pools of shared pages.
#pragma once

#include "dfa_serve.h"

namespace dfa {

constexpr int kTreeMaxTokens = 1024;  // nodes of a tree
constexpr int kTreeTile = 128;        // keys per tile
constexpr int kTreeRows = 128;        // query rows of a block
constexpr int kTreeMaxCtas = 160;     // (152 SMs)

struct TreePlanParams {
    CacheView c;
    const int32_t* q_lens;        // [B] or NULL
    const int32_t* parents;       // [B][T]
    int32_t T, words;
    uint32_t* mask;               // [B][T][words]
    int32_t* positions;           // [B][T]
};

struct TreeParams {
    CacheView c;
    Rows q;
    const int32_t* q_lens;        // [B] or NULL
    const uint32_t* mask;         // [B][T][words]
    int32_t words;
    int32_t Hq, G, T, o_fp32;
    uint32_t inv_T;               // 2^21 / T, rounded up
    int32_t row_groups;           // groups of query rows per key/value head
    int32_t line_blocks;          // blocks of a group; block c of group rg: c * row_groups + rg
    int32_t segment_cost;         // in tiles
    int32_t whole;                // segments are not cut
    float scale_log2;
    void* o;                      // [B, Hq, T, d]
    float* lse;                   // [B, Hq, T]
    int4* info;                   // [CTAs]: sequence, head and row group, CTAs that continue
                                  // it, nodes
    // [2 CTAs][rows]: what the sum is relative to (log2), what O is beyond that, sum
    float4* part_ndl;
    float* part_o;                // [2 CTAs][d / 4][rows][4]
    float* apart;                 // [2 CTAs][d / 4][rows][4]: O's earlier chains
    uint64_t timeout_ns;
};

constexpr int kCompactMaxParts = 4;  // blocks of a sequence's head and K or V

struct CompactParams {
    CacheView c;
    const int32_t* q_lens;        // [B] or NULL
    const int32_t* kept;          // [B][A]
    const int32_t* kept_lens;     // [B] or NULL
    int32_t T, A;
};

struct CopyParams {
    CacheView c;
    const int2* jobs;             // [max_jobs]: from page, to page
    const int32_t* info;          // info[0]: jobs
    int32_t max_jobs;
};

// Device view of a page pool (dfa_page_pool).
struct PoolView {
    int32_t* table;               // [B][max_pages]
    int32_t* held;                // [B]
    int32_t* refs;                // [npages]
    int32_t* seq_lens;            // [B]
    int64_t npages;
    int32_t B, max_pages, page_log2;
    DevStatus* status;
};

struct ForkParams {
    PoolView p;
    const int32_t* src;           // [B]
    int32_t* rows;                // [B][max_pages]: the new rows of the table
    int32_t* held;                // [B]
    int32_t* lens;                // [B]
};

struct ReserveParams {
    PoolView p;
    const int32_t* new_lens;      // [B] or NULL
    int32_t T, max_jobs;
    int32_t here;                 // the deciding block takes the pages, too
    int32_t lanes_log2;           // threads that look at a sequence's pages
    int2* jobs;
    int32_t* info;                // [4]
    int2* offset;                 // [B]: pages and jobs of the sequences before
    int32_t* last;                // [npages]: last sequence that writes the page
    int32_t* writers;             // [npages]
    int32_t* free;                // [npages]
};

cudaError_t launch_tree_plan(const TreePlanParams& p, cudaStream_t stream);
cudaError_t launch_decode_tree(const CUtensorMap& tk, const CUtensorMap& tv, TreeParams& p,
                               int num_sms, cudaStream_t stream);
cudaError_t launch_cache_compact(const CompactParams& p, cudaStream_t stream);
cudaError_t launch_cache_copy(const CopyParams& p, int num_sms, cudaStream_t stream);
cudaError_t launch_pages_fork(const ForkParams& p, cudaStream_t stream);
cudaError_t launch_pages_reserve(ReserveParams& p, cudaStream_t stream);
cudaError_t launch_pages_trim(const PoolView& p, cudaStream_t stream);

}  // namespace dfa
