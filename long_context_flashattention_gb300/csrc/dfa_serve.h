// dfa_serve.h -- plain-data structures shared by the host launchers and the
// kernels of rotary positions and of the paged key/value cache.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "dfa_params.h"

namespace dfa {

struct DevStatus;

// A rotary embedding as the kernels use it.  turn[t] is pair t's frequency as a
// 64-bit fraction of a full turn, so that (position * turn[t]) mod 2^64 is the
// reduced angle, in integer arithmetic: the reduction adds nothing to what the
// frequency itself, made in fp64, is off by (2^-51 of it at most).
struct RopeTable {
    uint64_t turn[64];
    float gain;
    int32_t half_layout;  // pairs (t, t + half) instead of (2t, 2t + 1)
    int32_t half;         // rot_dim / 2; 0: no rotation
};

// A row tensor [B, H, L, d] with contiguous features; strides in elements.
struct Rows {
    void* p;
    int64_t sb, sh, sl;
};

struct RopeRowsParams {
    RopeTable t;
    Rows x, out;
    int32_t B, H, d;
    int64_t L;
    int32_t inverse;
    int32_t heads;                // heads per work item
    const int32_t* positions;     // [B][L] or NULL
    DevMap map;
};

// Device view of a paged cache (dfa_paged_cache).
struct CacheView {
    void* k;
    void* v;
    float* k_scale;
    float* v_scale;
    const int32_t* table;
    const int32_t* seq_lens;
    int64_t npages, page_stride;  // page_stride in elements
    int32_t B, Hkv, d, page, page_log2, max_pages, e4m3;
    DevStatus* status;
};

struct AppendParams {
    CacheView c;
    RopeTable t;
    const int32_t* new_lens;      // [B] or NULL
    Rows k, v, q, q_out;
    int32_t T, Hq;
    int32_t pages;                // pages a sequence's new rows may touch
    // E4M3, page jobs: K or V rows of one page and `job_heads` heads, by
    // `job_threads` threads each
    int32_t job_heads, job_threads;
    uint32_t jobs;
    int32_t job_blocks;           // blocks with page jobs; the rest have row items
    // row items: one token, `item_heads` of its rows (q; and k, v of a bf16 cache)
    int32_t item_heads;
    uint32_t items;
};

struct GatherParams {
    CacheView c;
    int64_t pos0, L;
    void* k_out;
    void* v_out;
    int32_t page0, pages;         // pages [page0, page0 + pages) hold the rows
};

struct PagedParams {
    CacheView c;
    Rows q;
    const int32_t* q_lens;        // [B] or NULL
    int32_t Hq, G, T, causal, o_fp32;
    uint32_t inv_T;               // 2^21 / T, rounded up
    int32_t row_groups;           // groups of query rows per key/value head
    int32_t line_blocks;          // blocks of a group; block c of group rg: c * row_groups + rg
    int32_t segment_cost;         // in tiles
    int32_t whole;                // segments are not cut
    float scale_log2;
    void* o;                      // [B, Hq, T, d]
    float* lse;                   // [B, Hq, T]
    int4* info;                   // [CTAs]: sequence, head and row group, CTAs that continue it
    // [2 CTAs][rows]: what the sum is relative to (log2), what O is beyond that, sum
    float4* part_ndl;
    float* part_o;                // [2 CTAs][rows][d]
    uint64_t timeout_ns;
};

// Query rows that a decoding block works on at a time, and the most blocks.
constexpr int kPagedRows = 8, kPagedMaxRows = 16, kPagedMaxCtas = 512;
constexpr int kPagedTile = 64;    // keys per tile

cudaError_t launch_rope_rows(RopeRowsParams& p, int fp32, int num_sms, cudaStream_t stream);
cudaError_t launch_cache_append(AppendParams& p, int num_sms, cudaStream_t stream);
cudaError_t launch_cache_gather(const GatherParams& p, cudaStream_t stream);
cudaError_t launch_decode_paged(const CUtensorMap& tk, const CUtensorMap& tv,
                                PagedParams& p, int num_sms, cudaStream_t stream);

}  // namespace dfa
