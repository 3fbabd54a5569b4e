// dfa_paged.cu -- decoding attention over a paged key/value cache: the last few
// tokens of a ragged batch of sequences against their cached rows (FlashAttention
// glossary entry, the Flash-Decoding variant: the keys are split, partial results
// are merged by log-sum-exp rescaling).
//
// Method.  For a row q of a sequence, with keys k_j = s_j c_j (codes c_j times
// the scale s_j of their page and head) and values v_j = u_j w_j:
//   x_j = scale log2(e) s_j (q . c_j),   O = sum_j 2^(x_j - LSE) u_j w_j.
// The codes go into the matrix products as they are (e4m3 is exact in fp16); the
// key's scale multiplies the score, the value's scale its weight.  Weights are
// held as 2^(x_j + log2 u_j - M) with M the running maximum of the exponent, so
// that they stay in fp16's range whatever the scales are.  The exponent is rounded to
// fp32 like a score before M is taken off it, as M was when it was one of them: the
// difference is then exact and at most zero however large both are.  The sum of
// probabilities collects 2^(x_j - N) in fp32: N = M, and the weights over u_j are
// its terms, as long as u_j is in [2^-40, 2^40]; from the first page on whose
// scale is not (values near the type's ends, pages of zeros) N is the running
// maximum of x_j itself, and M is held as N + D: D is small, and large scores drop out
// of (x_j - N) + (log2 u_j - D).  O = 2^D (weighted sum) / (sum), D = 0 for M = N.
//
// What bounds it: HBM, up to 8 query rows a head (16 in bf16): a cached row is read once
// and meets G*T query rows, a few operations a byte.  The products are the 16x8x16 warp
// products, with the cache in the 16-row operand and 8 query rows (NB = 1) or 16 (NB = 2)
// in the other: S^T = K Q^T, O^T = V^T P^T.  With more rows the products and the
// conversions bound it; tcgen05 with 128 keys in M would serve there, and is not built.
//
// Work.  (sequence, head) segments of 64-key tiles form one line, cut by cost over
// a persistent grid whatever the lengths: a block's range covers whole segments,
// whose result it writes, and up to two cut ones, whose partials it leaves in the
// workspace for merge_kernel.  The lengths are read on the device, so a captured
// graph follows them.  A head with more than 16 query rows has several groups of
// them, and each group blocks of its own, cut alike: the groups' blocks read the same
// tiles at about the same time, out of L2.  Measured (4 sequences of 32K rows, 8 heads,
// bf16; 16, 32, 64, 128, 256 query rows, us): 90, 113, 195, 366, 709, where groups one
// behind the other on the line took 92, 162, 310, 604, 1182.  In 8 bits the products
// bound it, 58, 102, 191, 370, 725 either way.
//
// A block: warp 4 fetches pages by TMA into a ring of tiles (128- or 64-byte
// swizzle; the page numbers and scales of 32 pages are looked up at a time);
// warps 0-3 take 16 keys of every tile each, with a running maximum, sum and O
// of their own, joined at the segment's end.
//
// Measured (64 ragged sequences of up to 8192 rows, 8 heads of 128, 1.12 GB in
// bf16): bf16 167 us, 6.7 TB/s, 8-bit 93 us, 6.0 TB/s; with 16 query rows a head
// 175 and 117 us (twice the products for the bytes).  One 128K sequence of 32
// heads, 8-bit: 162 us, 6.6 TB/s.  About 10 us of each are fixed: the launch, the way to
// the first tile (lengths, page number, page), the last blocks' tail and the
// merge, which make up all of the 9.5 us of one sequence of 1000 rows.
//
// Rounding: weights for 8-bit cells as two fp16 terms (2^-22); as one (2^-11) for more
// than 8 query rows with a bf16 output (2^-8), where the products bound the kernel.
// Measured (one term, two; us): 64 ragged sequences, 16 rows 116, 132, 8 rows 91.3, 92.4;
// 128K x 32 heads 157.4, 158.6.  q for 8-bit cells as fp16 relative to a power of two of
// the row: exact but for elements below 2^-31 of its largest one, which are off by 2^-39 of
// that at most.  For bf16 cells q as it is and the weight as two bf16 terms (2^-16), since
// one would add as much error as the rounding of O.
#include <cfloat>

#include "dfa_serve.cuh"

namespace dfa {

namespace paged {

constexpr int kWarps = 4;                  // consumer warps
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kTile = kPagedTile;
// M is set kHead below the running maximum, and set anew when a weight exceeds 2^kTop.
// 8-bit cells have fp16 weights and use that type's range to its end (2^16): a weight
// has all its bits down to 2^-25 of the largest one, and half a step of those below is
// 2^-36 of it, so that the many small weights behind one large key add up to what they
// should.  Measured (kHead 7, 11, 13; 64 ragged sequences, 16 query rows, us): 130.8,
// 132.2, 133.6; with 8 rows no difference.
template <bool F8>
constexpr float kTop = F8 ? 15.f : 8.f;
template <bool F8>
constexpr float kHead = F8 ? 11.f : 0.f;
constexpr float kGrow = 8.f;               // the sum's own reference grows by 2^8 at least
constexpr float kNone = -FLT_MAX;          // running maximum before the first key
constexpr float kNear = 40.f;              // N = M while |log2 u_j| is at most this: the
                                           // terms are then 2^-80 or more of one another's
                                           // weights, far from fp32's ends
// Where no sequence can be longer than so many tiles, segments are not cut and
// there is nothing to merge.  Measured (GPU us cut, and whole; 1, 4, 8, 16 tiles): one
// sequence of 8 heads, 8-bit 7.8 7.0, 9.8 8.6, 9.4 10.7, 9.8 14.8; 64 sequences 10.7
// 9.9, 14.8 13.9, 18.5 20.1, 30.2 34.0; 16 of bf16 with 16 rows (2, 4, 8, 16 tiles)
// 11.5 9.9, 14.0 11.1, 15.6 13.7, 19.3 19.7.
constexpr int kWhole = 4;
constexpr float kNoPage = -1.f;            // in place of a key scale
constexpr float kLn2 = 0.69314718055994531f;

template <int D, bool F8, int NB>
struct Cfg {
    static constexpr int kRowBytes = D * (F8 ? 1 : 2);
    static constexpr int kPlanes = kRowBytes > 128 ? 2 : 1;  // boxes side by side
    static constexpr int kPlaneBytes = kRowBytes / kPlanes;  // 64 or 128: swizzle width
    static constexpr int kOperand = kTile * kRowBytes;       // K or V of a tile
    static constexpr int kStage = 2 * kOperand;
    static constexpr int kStages = kStage >= 32768 ? 2 : 49152 / kStage;
    static constexpr int kRows = 8 * NB;
    static constexpr int kPitch = D + 4;                     // floats of an O row in the join
    static constexpr int kJoin = kWarps * kRows * kPitch * 4;
    static constexpr int kQRows = kRows * D * 2;  // a segment's queries, two segments
    // What a segment costs a block beside its tiles, in tiles.  Measured (the batch
    // above; 1, 2, 3, 4, 5, 6): e4m3 91.4, 90.8, 90.9, 91.7 us; with 16 query rows 136,
    // 129, 126, 118, 115, 115; bf16 with 16 rows 177, 174, 174, 175.  256 sequences to
    // 1024 rows: 56.3, 52.6, 52.7, 54.4; 121, 106, 97.8, 89.9, 87.2, 87.7; 110, 99.7, 97.7,
    // 100.
    static constexpr int kSegmentCost = F8 && NB == 2 ? 5 : 2;
    // 16 query rows take their operand from shared memory: O takes its registers
    static constexpr int kQ = NB > 1 ? NB * (D / 16) * 32 * 8 : 0;
    static constexpr int kSmem = 1024 + kStages * kStage + kJoin + 2 * kQRows + kQ;
    // blocks of an SM that are resident together (registers and shared memory)
    static constexpr int kResident = NB == 1 && kStage < 32768 ? 3 : 2;
    static constexpr int kSteps = D / 16;                    // products over the features
};

// A run of tiles [tile0, tile0 + nt) of one segment: key/value head h, row group
// rg of sequence b, which has len rows, n queries and that many tiles.
struct Piece {
    int32_t b, h, rg, len, n;
    int32_t tile0, nt, tiles;
    long long w;      // the segment's first unit on the line
};

struct Shared {
    uint64_t full[8], empty[8];   // tiles
    uint64_t q_full[2], q_empty[2];
    uint64_t meet;                // of the consumer warps
    Piece run[2];                   // of the segments whose queries are there
    float4 scale[8][4];           // per stage and page: see page_scale
    // N, D and sums of the warps at a segment's end; two sets, since a warp may
    // end the next segment while another still reads this one's
    // (n: while D is not 0, a warp's entry is also where N is kept)
    float n[2][kWarps][kPagedMaxRows], d[2][kWarps][kPagedMaxRows], l[2][kWarps][kPagedMaxRows];
    float qf[2][8];               // NB = 2: score factors of the query rows
    long long warp_sum[kThreads / 32];
    long long w0, w1, base;       // the block's range; first unit of sequence b
    long long each, rest;         // units of a block; the first `rest` blocks have one more
    int32_t b, block;             // ..., and the block's place in its group
    uint32_t abort;
};

// A barrier of the consumer warps whose wait is bounded like the others; false:
// the block is giving up.
__device__ __forceinline__ bool meet(Shared& sh, uint32_t& phase, const WaitCtx& wctx)
{
    __syncwarp();
    if ((threadIdx.x & 31) == 0)
        mbar_arrive(&sh.meet);
    const bool ok = mbar_wait(&sh.meet, phase, wctx, 62);
    phase ^= 1;
    return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint64_t* bar,
                                            int c0, int c1, int c2, int c3)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2),
        "r"(c3)
        : "memory");
}

__device__ __forceinline__ void bulk_load_u32(uint32_t dst, const void* src, uint32_t bytes,
                                              uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
            "r"(dst),
        "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void mbar_expect(uint64_t* bar, uint32_t bytes)
{
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)),
                 "r"(bytes)
                 : "memory");
}

// D (16x8, fp32) += A (16x16) B (16x8), fp16 or bf16 operands
template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1)
{
    if (F16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, "
                     "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, "
                     "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// D = A B
template <bool F16>
__device__ __forceinline__ void mma16816_first(float (&d)[4], uint32_t a0, uint32_t a1,
                                               uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    if (F16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, "
                     "{%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                     : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, "
                     "{%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                     : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// transpose of an 8x8 matrix of 16-bit elements held one row per 4 lanes
__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}

__device__ __forceinline__ uint2 lds64(uint32_t a)
{
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}

// Byte offset of 16-byte chunk c of row r of a swizzled plane.
template <int PB>
__device__ __forceinline__ uint32_t chunk_at(uint32_t r, uint32_t c)
{
    return PB == 128 ? r * 128u + ((c ^ (r & 7u)) << 4) : r * 64u + ((c ^ ((r >> 1) & 3u)) << 4);
}

// Query row r of a key/value head: head of the group and token.
__device__ __forceinline__ void split_row(const PagedParams& p, int32_t r, int32_t& gh, int32_t& tq)
{
    gh = (int32_t)(((uint32_t)r * p.inv_T) >> 21);  // r / T: r below 2^11
    tq = r - gh * p.T;
}

// Tiles of a sequence with `n` queried tokens: at least one, so that rows
// without keys are written too.
__device__ __forceinline__ int32_t tiles_of(int32_t len, int32_t n)
{
    return n > 0 ? max(1, ceil_div(len, kTile)) : 0;
}

// a / b for a >= 0, b > 0, the short way where a has 32 bits
__device__ __forceinline__ long long divide(long long a, int32_t b)
{
    return a >> 32 ? a / b : (long long)((uint32_t)a / (uint32_t)b);
}

// The block of the group whose range has this unit.
__device__ __forceinline__ int block_of(const PagedParams& p, const Shared& sh, long long unit)
{
    const long long longer = sh.rest * (sh.each + 1);
    const long long c = unit < longer ? unit / (sh.each + 1) : sh.rest + (unit - longer) / sh.each;
    return (int)min(c, (long long)p.line_blocks - 1);
}

// The line that is cut: every segment takes p.segment_cost units (its queries, the join
// and the rows' output cost a block about that many tiles' time), then one unit
// per tile.  A cut inside the former puts the whole segment behind it.
//
// The producer's way along the block's range.  (Lengths that change while the
// kernel runs give results without meaning, but nothing worse: only this one
// warp goes by them, and every index that comes of them is checked.)
struct Walk : Piece {
    long long w1;     // end of the range
    bool fresh;       // tile0 is where the range begins

    __device__ __forceinline__ void start(const PagedParams& p, const Shared& sh, int32_t group)
    {
        w = sh.w0;
        w1 = sh.w1;
        b = sh.b;
        fresh = true;
        if (w >= w1)
            return;
        seq_rows(p.c, p.q_lens, p.T, b, len, n);
        tiles = tiles_of(len, n);
        const long long at = w - sh.base, unit = tiles + p.segment_cost;
        h = (int32_t)min(divide(at, (int32_t)unit), (long long)p.c.Hkv - 1);
        rg = group;
        const int32_t within = (int32_t)min(at - h * unit, unit - 1);
        tile0 = max(0, within - p.segment_cost);
        w -= within;  // the segment's first unit
        fresh = !p.whole || within == 0;  // else: begin with the next segment
    }
    __device__ __forceinline__ bool next(const PagedParams& p)
    {
        if (!fresh) {
            w += tiles + p.segment_cost;
            if (w >= w1)
                return false;
            tile0 = 0;
            if (++h == p.c.Hkv) {
                h = 0;
                do {
                    if (++b >= p.c.B)
                        return false;
                    seq_rows(p.c, p.q_lens, p.T, b, len, n);
                    tiles = tiles_of(len, n);
                } while (tiles == 0);
            }
        } else if (w >= w1) {
            return false;
        }
        fresh = false;
        nt = (int32_t)(p.whole ? tiles : min((long long)tiles, w1 - w - p.segment_cost)) - tile0;
        return nt > 0;  // (the last segment's beginning may lie in the range, its tiles behind)
    }
};

// The block's range of the line of tiles, and the sequence that it begins in.
template <int NB>
__device__ __forceinline__ void find_range(const PagedParams& p, Shared& sh)
{
    const int32_t per_seq = p.c.Hkv;
    const int32_t chunk = ceil_div(p.c.B, kThreads);
    // (up to 8 query rows are one group)
    const int32_t block = NB == 1 ? blockIdx.x : blockIdx.x / p.row_groups;
    if (threadIdx.x == 0) {
        sh.b = 0;
        sh.block = block;
        sh.base = 0;
    }
    const int32_t b0 = threadIdx.x * chunk, b1 = min(b0 + chunk, p.c.B);
    long long sum = 0;
    for (int32_t b = b0; b < b1; ++b) {
        int32_t len, n;
        seq_rows(p.c, p.q_lens, p.T, b, len, n);
        const int32_t tiles = tiles_of(len, n);
        sum += tiles ? (long long)(tiles + p.segment_cost) * per_seq : 0;
    }
    long long incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, incl, o);
        if ((threadIdx.x & 31) >= o)
            incl += x;
    }
    if ((threadIdx.x & 31) == 31)
        sh.warp_sum[threadIdx.x >> 5] = incl;
    __syncthreads();
    long long before = 0, total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < (threadIdx.x >> 5))
            before += sh.warp_sum[w];
        total += sh.warp_sum[w];
    }
    incl += before;
    const int32_t active = (int32_t)min((long long)p.line_blocks, total);
    const bool mine = block < active;  // then at least one unit
    const long long each = divide(total, max(active, 1)), rest = total - each * active;
    const long long w0 = mine ? each * block + min((long long)block, rest) : 0;
    const long long w1 = mine ? w0 + each + (block < rest ? 1 : 0) : 0;
    if (threadIdx.x == 0) {
        sh.w0 = w0;
        sh.w1 = w1;
        sh.each = each;
        sh.rest = rest;
    }
    if (w0 < w1 && incl - sum <= w0 && w0 < incl) {
        long long base = incl - sum;
        for (int32_t b = b0; b < b1; ++b) {
            int32_t len, n;
            seq_rows(p.c, p.q_lens, p.T, b, len, n);
            const int32_t tiles = tiles_of(len, n);
            const long long t = tiles ? (long long)(tiles + p.segment_cost) * per_seq : 0;
            if (w0 < base + t) {
                sh.b = b;
                sh.base = base;
                break;
            }
            base += t;
        }
    }
    __syncthreads();
}

// What a group of 16 keys needs of its page's scales s (K) and u (V): s, log2 u, 1 / u.
template <bool F8>
__device__ __forceinline__ float4 page_scale(bool there, float s, float u)
{
    if (!there)
        return make_float4(kNoPage, 0.f, 0.f, 0.f);
    if (!F8)
        return make_float4(1.f, 0.f, 1.f, 0.f);
    // exponent and significand apart: exact for a power of two
    const uint32_t bits = __float_as_uint(u);
    const int e = (int)((bits >> 23) & 0xffu);
    const float lu = e == 255 ? u : (float)max(e - 127, -126) +
                                        log2f(__uint_as_float((bits & 0x7fffffu) | (127u << 23)));
    return make_float4(s, lu, ex2(-lu), 0.f);
}

// The producer warp: queries of a segment, then its tiles.  Every wait it has for
// itself (lengths, page numbers, scales of the next segment) begins while tiles
// of this one are still to be fetched.
template <int D, bool F8, int NB>
__device__ __forceinline__ void produce(const PagedParams& p, Shared& sh, uint32_t ring,
                                        uint32_t q_rows, const CUtensorMap& tk,
                                        const CUtensorMap& tv, const WaitCtx& wctx)
{
    using C = Cfg<D, F8, NB>;
    const int lane = threadIdx.x & 31;
    const int32_t page = p.c.page;
    const int32_t box_rows = min(page, kTile);
    const int32_t per_tile = kTile / box_rows;  // boxes of a tile
    uint32_t st = 0, phase = 0, seg = 0;
    Walk wk;
    wk.start(p, sh, NB == 1 ? 0 : blockIdx.x - sh.block * p.row_groups);
    bool more = wk.next(p);
    // Table entry of this lane's page of the 32 from page `win` on; -1: none.
    auto entry = [&](const Walk& x, int32_t win) {
        const int32_t end = ceil_div(min(x.len, (x.tile0 + x.nt) * kTile), page);
        return win + lane < end ? page_entry(p.c, x.b, win + lane) : -1;
    };
    int32_t next_id = more ? entry(wk, (wk.tile0 * kTile) >> p.c.page_log2) : -1;
    for (; more; ++seg) {
        const int32_t h = wk.h;
        const int32_t pages_end =
            ceil_div(min(wk.len, (wk.tile0 + wk.nt) * kTile), page);  // of this run
        int32_t win = (wk.tile0 * kTile) >> p.c.page_log2, id = next_id;
        float ks = 1.f, vs = 1.f;
        auto check_window = [&] {  // the lane's page, and its scales on their way
            if (win + lane >= pages_end || !is_page(p.c, wk.b, id)) {
                id = -1;
            } else if (F8) {
                const int64_t at = (int64_t)id * p.c.Hkv + h;
                ks = __ldcg(p.c.k_scale + at);  // (an append may have just raised them)
                vs = __ldcg(p.c.v_scale + at);
            }
        };
        check_window();
        auto fetch_queries = [&] {
            const uint32_t qb = seg & 1;
            const bool ok = mbar_wait(&sh.q_empty[qb], (seg / 2 + 1) & 1, wctx, 51);
            if (!__all_sync(0xffffffffu, ok))
                return false;
            const int32_t r = wk.rg * C::kRows + lane;
            int32_t gh, tq;
            split_row(p, r, gh, tq);
            const bool there = lane < C::kRows && r < p.G * p.T && tq < wk.n;
            const uint32_t rows = __popc(__ballot_sync(0xffffffffu, there));
            if (lane == 0) {
                sh.run[qb] = wk;
                mbar_expect(&sh.q_full[qb], rows * (D * 2));
            }
            __syncwarp();
            if (there)
                bulk_load_u32(q_rows + qb * C::kQRows + lane * (D * 2),
                              (const __nv_bfloat16*)p.q.p + wk.b * p.q.sb +
                                  (int64_t)(h * p.G + gh) * p.q.sh + (int64_t)tq * p.q.sl,
                              D * 2, &sh.q_full[qb]);
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sh.q_full[qb]);
            return true;
        };
        Walk nx = wk;
        bool more_next = false;
        const int32_t look = min(wk.nt - 1, C::kStages - 1);
        for (int32_t i = 0; i < wk.nt; ++i) {
            const int32_t key0 = (wk.tile0 + i) * kTile;
            const int32_t p0 = key0 >> p.c.page_log2;
            if (p0 >= win + 32) {
                win = p0;
                id = entry(wk, win);
                check_window();
            }
            // (passes at once in the first round: the phase before the barrier's first)
            const bool ok = mbar_wait(&sh.empty[st], phase ^ 1, wctx, 50);
            if (!__all_sync(0xffffffffu, ok))
                return;
            const int src = p0 - win + lane;  // lanes below per_tile: their box's page
            const int32_t my = __shfl_sync(0xffffffffu, id, src & 31);
            const bool load = lane < per_tile && p0 + lane < pages_end && my >= 0;
            const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, load));
            if (lane == 0)
                mbar_expect(&sh.full[st], boxes * (2 * box_rows * C::kRowBytes));
            __syncwarp();
            if (load) {
                const uint32_t dst = ring + st * C::kStage + lane * box_rows * C::kPlaneBytes;
                const int row = key0 & (page - 1);  // 0 unless a page holds several tiles
#pragma unroll
                for (int pl = 0; pl < C::kPlanes; ++pl) {
                    const uint32_t d2 = dst + pl * kTile * C::kPlaneBytes;
                    tma_load_4d(d2, &tk, &sh.full[st], pl * 64, row, h, my);
                    tma_load_4d(d2 + C::kOperand, &tv, &sh.full[st], pl * 64, row, h, my);
                }
            }
            // the scales last: they may still be on their way
            const float my_ks = __shfl_sync(0xffffffffu, ks, src & 31);
            const float my_vs = __shfl_sync(0xffffffffu, vs, src & 31);
            if (lane < per_tile)
                sh.scale[st][lane] = page_scale<F8>(load, my_ks, my_vs);
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sh.full[st]);
            if (++st == C::kStages) {
                st = 0;
                phase ^= 1;
            }
            if (i == 0 && !fetch_queries())
                return;
            if (i == look) {
                more_next = nx.next(p);
                next_id = more_next ? entry(nx, (nx.tile0 * kTile) >> p.c.page_log2) : -1;
            }
        }
        wk = nx;
        more = more_next;
    }
    // no more runs
    const bool ok = mbar_wait(&sh.q_empty[seg & 1], (seg / 2 + 1) & 1, wctx, 52);
    if (__all_sync(0xffffffffu, ok) && lane == 0) {
        sh.run[seg & 1].nt = 0;
        mbar_arrive(&sh.q_full[seg & 1]);
    }
}

template <bool TRANS>
__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4])
{
    if (TRANS)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(addr)
                     : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(addr)
                     : "memory");
}

// V of a warp's 16 keys as 16x16 operands V^T (a0, a1: keys 2t, 2t+1; a2, a3: keys
// 2t+8, 2t+9), tile by tile of 16 features.  clip(n): the keys from the group's
// n-th on are zero.
//
// bf16: the matrix loads transpose; tile m has features 16m + g (a0, a2) and
// 16m + 8 + g (a1, a3).
template <typename C, bool F8>
struct Values {
    uint32_t base, key_, keep[2];

    __device__ __forceinline__ void load(uint32_t vt, uint32_t row)
    {
        const int lane = threadIdx.x & 31;
        base = vt;
        key_ = row + (lane & 7) + (lane >> 4) * 8;
    }
    __device__ __forceinline__ void clip(int upto)
    {
        const int t = threadIdx.x & 3;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            keep[i] = (2 * t + 8 * i < upto ? 0xffffu : 0u) |
                      (2 * t + 8 * i + 1 < upto ? 0xffff0000u : 0u);
    }
    template <bool CLIPPED>
    __device__ __forceinline__ void tile(int m, uint32_t (&a)[4]) const
    {
        const uint32_t c = 2 * m + ((threadIdx.x >> 3) & 1);  // 16-byte chunk of the row
        const uint32_t plane = base + (c >> 3) * kTile * C::kPlaneBytes;
        ldmatrix4<true>(plane + chunk_at<128>(key_, c & 7), a);
        if (CLIPPED) {
            a[0] &= keep[0], a[1] &= keep[0];
            a[2] &= keep[1], a[3] &= keep[1];
        }
    }
    static __device__ __forceinline__ bool not_finite(uint32_t w)
    {
        return (w & 0x7f800000u) == 0x7f800000u || (w & 0x7f80u) == 0x7f80u;
    }
};

// e4m3: a lane reads 16 (d = 128) or 8 features of four keys and turns them to
// fp16; tile m has its features 2m (a0, a2) and 2m + 1 (a1, a3).
template <typename C>
struct Values<C, true> {
    static constexpr int W = C::kPlaneBytes / 32;  // words per key
    uint32_t w[4][W];

    __device__ __forceinline__ void load(uint32_t vt, uint32_t row)
    {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int key = 2 * t + (k & 1) + (k >> 1) * 8;
            if (W == 4) {
                const uint4 x = lds128(vt + chunk_at<C::kPlaneBytes>(row + key, g));
                w[k][0] = x.x, w[k][1] = x.y;
                w[k][W - 2] = x.z, w[k][W - 1] = x.w;
            } else {
                const uint2 x =
                    lds64(vt + chunk_at<C::kPlaneBytes>(row + key, g >> 1) + (g & 1) * 8);
                w[k][0] = x.x, w[k][1] = x.y;
            }
        }
    }
    __device__ __forceinline__ void clip(int upto)
    {
        const int t = threadIdx.x & 3;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (2 * t + (k & 1) + (k >> 1) * 8 >= upto)
#pragma unroll
                for (int i = 0; i < W; ++i)
                    w[k][i] = 0u;
    }
    template <bool CLIPPED>
    __device__ __forceinline__ void tile(int m, uint32_t (&a)[4]) const
    {
        const uint32_t sel = (m & 1) ? 0x7362 : 0x5140;  // features 2m, 2m+1 of two keys
        const uint32_t x = __byte_perm(w[0][m / 2], w[1][m / 2], sel);
        const uint32_t y = __byte_perm(w[2][m / 2], w[3][m / 2], sel);
        a[0] = e4m3x2_half2(x & 0xffffu);
        a[1] = e4m3x2_half2(x >> 16);
        a[2] = e4m3x2_half2(y & 0xffffu);
        a[3] = e4m3x2_half2(y >> 16);
    }
    static __device__ __forceinline__ bool not_finite(uint32_t h)  // of a pair of fp16
    {
        return (h & 0x7c000000u) == 0x7c000000u || (h & 0x7c00u) == 0x7c00u;
    }
};

// 8 query rows in shared memory as the products' operand (16 features a step, two
// words a lane), rows that are not `there` (lane: row g) as zeros.  Returns the
// factor of row g's scores.  e4m3: as fp16 relative to a power of two, at which the
// row's largest element is next to fp16's end, in the order in which the lanes hold K's
// features.
template <int D, bool F8>
__device__ __forceinline__ float load_queries(uint32_t rows, bool there, float scale_log2,
                                              uint32_t (&q)[D / 16][2])
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    if constexpr (!F8) {
#pragma unroll
        for (int s = 0; s < D / 16; s += 2) {
            // chunks 2s .. 2s+3 of the rows
            uint32_t r[4];
            ldmatrix4<false>(rows + (lane & 7) * (D * 2) + (2 * s + (lane >> 3)) * 16, r);
            q[s][0] = there ? r[0] : 0u, q[s][1] = there ? r[1] : 0u;
            q[s + 1][0] = there ? r[2] : 0u, q[s + 1][1] = there ? r[3] : 0u;
        }
        return scale_log2;
    } else {
#pragma unroll
        for (int s = 0; s < D / 16; s += 2) {
            uint4 x = lds128(rows + g * (D * 2) + t * (D / 2) + s * 8);
            if (!there)
                x = make_uint4(0, 0, 0, 0);
            q[s][0] = x.x, q[s][1] = x.y;
            q[s + 1][0] = x.z, q[s + 1][1] = x.w;
        }
        float amax = 0.f;
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
#pragma unroll
            for (int k = 0; k < 2; ++k)
                amax = fmaxf(amax, fmaxf(fabsf(bf16lo(q[s][k])), fabsf(bf16hi(q[s][k]))));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        // the largest element to [2^14, 2^15): those down to 2^-31 of it stay exact
        const int e = min(max((int)(__float_as_uint(amax) >> 23) - 127, -100), 126) - 14;
        const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
#pragma unroll
            for (int k = 0; k < 2; ++k)
                q[s][k] = pack_half2(bf16lo(q[s][k]) * inv, bf16hi(q[s][k]) * inv);
        return scale_log2 * __uint_as_float((uint32_t)(127 + e) << 23);
    }
}

// Features f..f+3 of an output row, and its LSE: o is relative to 2^(nx + dx), L to 2^nx.
template <int D, bool F8>
__device__ __forceinline__ void write_row(const PagedParams& p, int64_t at, int f, float nx,
                                          float dx, float L, float4 o)
{
    // 2^dx in two halves: it may be below fp32's range where o makes up for it
    const float half = F8 ? ex2(0.5f * dx) : 1.f;
    const float inv = L == 0.f ? 0.f : half / L;  // (NaN stays NaN)
    o.x *= inv, o.y *= inv, o.z *= inv, o.w *= inv;
    if (F8)
        o.x *= half, o.y *= half, o.z *= half, o.w *= half;
    if (p.o_fp32)
        *reinterpret_cast<float4*>((float*)p.o + at * D + f) = o;
    else
        *reinterpret_cast<uint2*>((__nv_bfloat16*)p.o + at * D + f) =
            make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
    if (f == 0)
        p.lse[at] = L == 0.f ? -INFINITY : (nx + log2f(L)) * kLn2;
}

template <int D, bool F8, int NB, bool TWO_TERMS>
__device__ __forceinline__ void consume(const PagedParams& p, Shared& sh, uint32_t ring,
                                        float* join, uint32_t q_rows, uint2* qs,
                                        const WaitCtx& wctx)
{
    using C = Cfg<D, F8, NB>;
    constexpr int kMt = D / 16;                   // O^T tiles of 16 features
    constexpr int kChunks = C::kPlaneBytes / 64;  // e4m3: K chunks per lane
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int32_t page = p.c.page;
    const int sc_at = page < kTile ? warp * 16 / page : 0;
    const int32_t R = p.G * p.T;
    uint32_t st = 0, phase = 0, met = 0;
    int4 info = make_int4(0, 0, 0, 0);
    for (uint32_t seg = 0;; ++seg) {
        bool ok = mbar_wait(&sh.q_full[seg & 1], (seg / 2) & 1, wctx, 61);
        if (!__all_sync(0xffffffffu, ok))
            return;
        const Piece wk = sh.run[seg & 1];
        if (wk.nt == 0)
            break;
        const int32_t h = wk.h, r0 = NB == 1 ? 0 : wk.rg * C::kRows;
        const int32_t len = wk.len, n = wk.n;
        // ---- queries: rows g of each block of 8, this lane's features
        uint32_t q[C::kSteps][2];  // NB = 1: the operand itself
        uint64_t rf[NB];           // score factors of rows 2t, 2t+1
        int32_t lim[NB][2];        // last visible key of rows 2t, 2t+1
        int32_t tok[NB][2];
        if (NB == 1 || warp < NB) {
            const int nb = NB == 1 ? 0 : warp;
            int32_t gh, tq;
            split_row(p, r0 + nb * 8 + g, gh, tq);
            const float f =
                load_queries<D, F8>(q_rows + (seg & 1) * C::kQRows + nb * 8 * (D * 2),
                                    r0 + nb * 8 + g < R && tq < n, p.scale_log2, q);
            if (NB == 1) {
                rf[0] = f2pack(__shfl_sync(0xffffffffu, f, 2 * t * 4),
                               __shfl_sync(0xffffffffu, f, (2 * t + 1) * 4));
            } else {
#pragma unroll
                for (int s = 0; s < C::kSteps; ++s)
                    qs[(nb * C::kSteps + s) * 32 + lane] = make_uint2(q[s][0], q[s][1]);
                if (t == 0)
                    sh.qf[nb][g] = f;
            }
        }
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&sh.q_empty[seg & 1]);
        if (NB > 1 && !meet(sh, met, wctx))
            return;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            if (NB > 1)
                rf[nb] = f2pack(sh.qf[nb][2 * t], sh.qf[nb][2 * t + 1]);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int32_t rr = r0 + nb * 8 + 2 * t + k;
                int32_t gh, tq;
                split_row(p, rr, gh, tq);
                tok[nb][k] = rr < R ? tq : n;
                lim[nb][k] = p.causal ? len - n + min(tok[nb][k], n - 1) : len - 1;
            }
        }
        // keys up to all_see are visible to every row, keys from len on to none
        const int32_t all_see = p.causal ? len - n : len - 1;
        float O[NB][kMt][4], M[NB][2], l[NB][2];
        bool wide = false;  // N has left M: M[][] is D, and N in shared memory
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                M[nb][k] = kNone;
                l[nb][k] = 0.f;
            }
#pragma unroll
            for (int m = 0; m < kMt; ++m)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    O[nb][m][k] = 0.f;
        }
        // ---- the run's tiles
        for (int32_t i = 0; i < wk.nt; ++i) {
            ok = mbar_wait(&sh.full[st], phase, wctx, 60);
            if (!__all_sync(0xffffffffu, ok))
                return;
            const int32_t base = (wk.tile0 + i) * kTile + warp * 16;  // the warp's 16 keys
            const float4 sc = sh.scale[st][sc_at];
            if (base < len && sc.x != kNoPage) {
                const uint32_t kt = ring + st * C::kStage;
                const uint32_t vt = kt + C::kOperand;
                const uint32_t row = warp * 16;
                // S^T = K Q^T; two sums, so that half the products are independent
                float acc[NB][2][4];
                auto product = [&](int s, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        const uint2 b = NB == 1 ? make_uint2(q[s][0], q[s][1])
                                                : qs[(nb * C::kSteps + s) * 32 + lane];
                        if (s < 2)
                            mma16816_first<F8>(acc[nb][s & 1], a0, a1, a2, a3, b.x, b.y);
                        else
                            mma16816<F8>(acc[nb][s & 1], a0, a1, a2, a3, b.x, b.y);
                    }
                };
                if (F8) {
#pragma unroll
                    for (int c = 0; c < kChunks; ++c) {
                        const uint4 x =
                            lds128(kt + chunk_at<C::kPlaneBytes>(row + g, t * kChunks + c));
                        const uint4 y =
                            lds128(kt + chunk_at<C::kPlaneBytes>(row + g + 8, t * kChunks + c));
                        const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
                        const uint32_t yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            product(c * 4 + j, e4m3x2_half2(xw[j] & 0xffffu),
                                    e4m3x2_half2(yw[j] & 0xffffu), e4m3x2_half2(xw[j] >> 16),
                                    e4m3x2_half2(yw[j] >> 16));
                    }
                } else {
#pragma unroll
                    for (int s = 0; s < C::kSteps; ++s) {
                        const uint32_t plane = kt + (s / 4) * kTile * C::kPlaneBytes;
                        uint32_t a[4];
                        ldmatrix4<false>(plane + chunk_at<128>(row + (lane & 15),
                                                               (2 * s + (lane >> 4)) & 7),
                                         a);
                        product(s, a[0], a[1], a[2], a[3]);
                    }
                }
                const bool masked = base + 15 > all_see;  // some row does not see some key
                bool apart = false;  // non-finite V that some rows do not see
                Values<C, F8> v;
                if (masked && p.causal && n > 1) {
                    v.load(vt, row);
                    v.clip(len - base);
#pragma unroll
                    for (int m = 0; m < kMt; ++m) {
                        uint32_t a[4];
                        v.template tile<true>(m, a);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            apart |= v.not_finite(a[k]);
                    }
                    apart = __any_sync(0xffffffffu, apart);
                }
                float* own_n = sh.n[seg & 1][warp];
                if (F8 && __builtin_expect(!wide && !(fabsf(sc.y) <= kNear), 0)) {
                    wide = true;
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        if (g == 0)
                            *reinterpret_cast<float2*>(own_n + nb * 8 + 2 * t) =
                                make_float2(M[nb][0], M[nb][1]);
                        M[nb][0] = M[nb][1] = 0.f;
                    }
                    __syncwarp();
                }
                uint32_t pt[NB][2], pr[NB][2];  // P^T in two terms
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    // Rows 2t and 2t+1 of a pair, key g in x[0], x[1], key g + 8 in x[2], x[3].
                    const uint64_t factor = F8 ? f2mul(rf[nb], f2pack(sc.x, sc.x)) : rf[nb];
                    uint64_t dot[2];
                    float x[4], w[4];
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        dot[k] = f2add(f2pack(acc[nb][0][2 * k], acc[nb][0][2 * k + 1]),
                                       f2pack(acc[nb][1][2 * k], acc[nb][1][2 * k + 1]));
                    // x = score + lu - (m0, m1), the former rounded first
                    auto exponents = [&](float lu, float m0, float m1) {
                        const uint64_t off = f2pack(-m0, -m1);
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint64_t sum = F8 ? f2fma(dot[k], factor, f2pack(lu, lu))
                                                    : f2mul(dot[k], factor);
                            f2unpack(f2add(sum, off), x[2 * k], x[2 * k + 1]);
                        }
                        if (masked)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (base + g + 8 * (k >> 1) > lim[nb][k & 1])
                                    x[k] = -INFINITY;
                    };
                    // does any x exceed a bound?
                    auto exceeds = [&](float bound) {
                        return __any_sync(0xffffffffu,
                                          fmax3(x[0], x[1], fmaxf(x[2], x[3])) > bound);
                    };
                    // the rows' largest x
                    auto largest = [&](float(&mx)[2]) {
                        mx[0] = fmaxf(x[0], x[2]), mx[1] = fmaxf(x[1], x[3]);
#pragma unroll
                        for (int k = 0; k < 2; ++k)
#pragma unroll
                            for (int o = 4; o < 32; o <<= 1)
                                mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], o));
                    };
                    // M (or D) up to what the largest x asks for, O (and the sum) with it
                    auto raise = [&](const float(&mx)[2]) {
                        float f[2];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const float mn = fmaxf(M[nb][k], mx[k] - kHead<F8>);
                            f[k] = ex2(M[nb][k] - mn);
                            M[nb][k] = mn;
                            if (!F8 || !wide)
                                l[nb][k] *= f[k];
                        }
#pragma unroll
                        for (int m = 0; m < kMt; ++m)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                O[nb][m][k] *= f[k & 1];
                    };
                    float mx[2];
                    if (F8 && __builtin_expect(wide, 0)) {
                        float2* at = reinterpret_cast<float2*>(own_n + nb * 8 + 2 * t);
                        float2 N = *at;
                        exponents(0.f, N.x, N.y);
                        if (exceeds(kGrow)) {
                            exponents(0.f, 0.f, 0.f);
                            largest(mx);
                            mx[0] = fmaxf(N.x, mx[0]), mx[1] = fmaxf(N.y, mx[1]);
                            l[nb][0] *= ex2(N.x - mx[0]), l[nb][1] *= ex2(N.y - mx[1]);
                            M[nb][0] += N.x - mx[0], M[nb][1] += N.y - mx[1];
                            N = make_float2(mx[0], mx[1]);
                            __syncwarp();
                            if (g == 0)
                                *at = N;
                            exponents(0.f, N.x, N.y);
                        }
                        __syncwarp();
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            l[nb][k & 1] += ex2(x[k]);
                            x[k] += sc.y;
                        }
                        largest(mx);
                        if (__any_sync(0xffffffffu, mx[0] - M[nb][0] > kTop<F8> ||
                                                        mx[1] - M[nb][1] > kTop<F8>))
                            raise(mx);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            w[k] = ex2(x[k] - M[nb][k & 1]);
                    } else {
                        exponents(sc.y, M[nb][0], M[nb][1]);
                        if (exceeds(kTop<F8>)) {
                            exponents(sc.y, 0.f, 0.f);
                            largest(mx);
                            raise(mx);
                            exponents(sc.y, M[nb][0], M[nb][1]);
                            // kHead is rounded, too, where M is large (NaN stays NaN)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                x[k] = x[k] > kTop<F8> ? kTop<F8> : x[k];
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            w[k] = ex2(x[k]);
                            l[nb][k & 1] =
                                F8 ? fmaf(w[k], sc.z, l[nb][k & 1]) : l[nb][k & 1] + w[k];
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        if (F8) {
                            const uint32_t hi = pack_half2(w[2 * k], w[2 * k + 1]);
                            pt[nb][k] = transpose8(hi);
                            if (TWO_TERMS) {
                                const float2 y =
                                    __half22float2(*reinterpret_cast<const __half2*>(&hi));
                                pr[nb][k] =
                                    transpose8(pack_half2(w[2 * k] - y.x, w[2 * k + 1] - y.y));
                            }
                        } else {
                            const uint32_t hi = pack_bf16x2(w[2 * k], w[2 * k + 1]);
                            const uint32_t lo =
                                pack_bf16x2(w[2 * k] - bf16lo(hi), w[2 * k + 1] - bf16hi(hi));
                            pt[nb][k] = transpose8(hi);
                            pr[nb][k] = transpose8(lo);
                        }
                    }
                }
                // O^T += V^T P^T
                auto weigh = [&](int nb, float(&d)[4], const uint32_t(&a)[4]) {
                    mma16816<F8>(d, a[0], a[1], a[2], a[3], pt[nb][0], pt[nb][1]);
                    if (TWO_TERMS)
                        mma16816<F8>(d, a[0], a[1], a[2], a[3], pr[nb][0], pr[nb][1]);
                };
                if (!masked) {
                    v.load(vt, row);
#pragma unroll
                    for (int m = 0; m < kMt; ++m) {
                        uint32_t a[4];
                        v.template tile<false>(m, a);
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
                            weigh(nb, O[nb][m], a);
                    }
                } else {
                    // V of keys behind the end is not ours.  And a NaN or an infinity
                    // times a weight of zero would reach rows that do not see it:
                    // then one token at a time, with the values behind its position
                    // taken out.
                    for (int32_t tt = apart ? 0 : n - 1; tt < n; ++tt) {
                        v.load(vt, row);
                        v.clip((apart ? len - n + tt + 1 : len) - base);
#pragma unroll
                        for (int m = 0; m < kMt; ++m) {
                            uint32_t a[4];
                            v.template tile<true>(m, a);
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb) {
                                float d[4] = {O[nb][m][0], O[nb][m][1], O[nb][m][2], O[nb][m][3]};
                                weigh(nb, d, a);
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    if (!apart || tok[nb][k & 1] == tt)
                                        O[nb][m][k] = d[k];
                            }
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sh.empty[st]);
            if (++st == C::kStages) {
                st = 0;
                phase ^= 1;
            }
        }
        // ---- join the warps: common references, rescaled sums and O
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1)
                    l[nb][k] += __shfl_xor_sync(0xffffffffu, l[nb][k], o);
                if (g == 0) {
                    sh.l[seg & 1][warp][nb * 8 + 2 * t + k] = l[nb][k];
                    if (!F8 || !wide)
                        sh.n[seg & 1][warp][nb * 8 + 2 * t + k] = M[nb][k];
                    if (F8)
                        sh.d[seg & 1][warp][nb * 8 + 2 * t + k] = wide ? M[nb][k] : 0.f;
                }
            }
        if (!meet(sh, met, wctx))
            return;
        // N and D of all warps together, and what a warp's O is multiplied by
        const auto& ns = sh.n[seg & 1];
        const auto& ds = sh.d[seg & 1];
        auto common = [&](int r, float& nx, float& dx) {
            nx = ns[0][r];
#pragma unroll
            for (int w = 1; w < kWarps; ++w)
                nx = fmaxf(nx, ns[w][r]);
            dx = 0.f;
            if (F8) {
                dx = (ns[0][r] - nx) + ds[0][r];
#pragma unroll
                for (int w = 1; w < kWarps; ++w)
                    dx = fmaxf(dx, (ns[w][r] - nx) + ds[w][r]);
            }
        };
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int r = nb * 8 + 2 * t + k;
                float nx, dx;
                common(r, nx, dx);
                const float f = ex2((ns[warp][r] - nx) + ((F8 ? ds[warp][r] : 0.f) - dx));
                if (r0 + r < R) {
                    float* dst = join + (warp * C::kRows + r) * C::kPitch;
#pragma unroll
                    for (int m = 0; m < kMt; ++m) {
                        if (F8) {  // features 2m, 2m + 1 of the lane's kMt * 2
                            if (m % 2 == 0)
                                *reinterpret_cast<float4*>(dst + g * (2 * kMt) + 2 * m) =
                                    make_float4(O[nb][m][k] * f, O[nb][m][2 + k] * f,
                                                O[nb][m + 1][k] * f, O[nb][m + 1][2 + k] * f);
                        } else {
                            dst[16 * m + g] = O[nb][m][k] * f;
                            dst[16 * m + 8 + g] = O[nb][m][2 + k] * f;
                        }
                    }
                }
            }
        if (!meet(sh, met, wctx))
            return;
        // ---- rows of the segment: D/4 threads each
        constexpr int kPerRow = D / 4;
        const bool whole = wk.nt == wk.tiles;
        const int64_t slot = 2 * (int64_t)blockIdx.x + (wk.tile0 == 0 ? 1 : 0);
        for (int r = threadIdx.x / kPerRow; r < C::kRows && r0 + r < R;
             r += 32 * kWarps / kPerRow) {
            const int f = threadIdx.x % kPerRow * 4;
            float nx, dx, L = 0.f;
            common(r, nx, dx);
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                L += sh.l[seg & 1][w][r] * ex2(ns[w][r] - nx);
                const float4 y = *reinterpret_cast<const float4*>(
                    join + (w * C::kRows + r) * C::kPitch + f);
                o.x += y.x, o.y += y.y, o.z += y.z, o.w += y.w;
            }
            if (!whole) {
                if (f == 0)
                    p.part_ndl[slot * C::kRows + r] = make_float4(nx, dx, L, 0.f);
                *reinterpret_cast<float4*>(p.part_o + (slot * C::kRows + r) * D + f) = o;
                continue;
            }
            int32_t gh, tq;
            split_row(p, r0 + r, gh, tq);
            if (tq >= n)
                continue;
            const int64_t at = ((int64_t)wk.b * p.Hq + h * p.G + gh) * p.T + tq;
            write_row<D, F8>(p, at, f, nx, dx, L, o);
        }
        if (!whole && wk.tile0 == 0) {
            // the group's blocks after this one that hold the rest: up to the last tile's
            const long long last = wk.w + p.segment_cost + wk.tiles - 1;
            info = make_int4(wk.b, NB == 1 ? wk.h : wk.h * p.row_groups + wk.rg,
                             block_of(p, sh, last) - sh.block, n);
        }
    }
    if (threadIdx.x == 0)
        p.info[blockIdx.x] = info;
}

template <int D, bool F8, int NB, bool TWO_TERMS>
__global__ void __launch_bounds__(kThreads, Cfg<D, F8, NB>::kResident)
    decode_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                  const __grid_constant__ PagedParams p)
{
    using C = Cfg<D, F8, NB>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Shared sh;
    const uint32_t ring = (smem_u32(smem_raw) + 1023) & ~1023u;
    float* join = reinterpret_cast<float*>(smem_raw + (ring - smem_u32(smem_raw)) +
                                           C::kStages * C::kStage);
    const uint32_t q_rows = smem_u32(join) + C::kJoin;
    uint2* qs = reinterpret_cast<uint2*>(join + (C::kJoin + 2 * C::kQRows) / 4);
    if (threadIdx.x == 0) {
        sh.abort = 0;
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&sh.full[s], 1);
            mbar_init(&sh.empty[s], kWarps);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sh.q_full[s], 1);
            mbar_init(&sh.q_empty[s], kWarps);
        }
        mbar_init(&sh.meet, kWarps);
        fence_barrier_init();
        prefetch_tmap(&tk);
        prefetch_tmap(&tv);
    }
    cudaGridDependencySynchronize();            // (what the kernel before it wrote)
    cudaTriggerProgrammaticLaunchCompletion();  // merge_kernel's blocks may be launched
    if (threadIdx.x == 0)
        p.info[blockIdx.x] = make_int4(0, 0, 0, 0);  // for a block that gives up
    find_range<NB>(p, sh);  // also orders the barriers' initialisation
    const WaitCtx wctx{&sh.abort, p.c.status, p.timeout_ns};
    if (threadIdx.x >= 32 * kWarps) {
        produce<D, F8, NB>(p, sh, ring, q_rows, tk, tv, wctx);
        if (*wctx.abort_flag) {
            // let copies in flight land before the block's shared memory goes
            const uint64_t t0 = globaltimer_ns();
            while (globaltimer_ns() - t0 < 2000000ull) {
            }
        }
    } else {
        consume<D, F8, NB, TWO_TERMS>(p, sh, ring, join, q_rows, qs, wctx);
    }
}

// Rows of the segments that several blocks share: block c holds such a segment's
// beginning, the info[c].z blocks of its group after it the rest.  One warp a row; where most
// segments have many partials (a long sequence with few heads) a block a row.
template <int D, bool F8, int ROWS, bool BLOCK_A_ROW>
__global__ void __launch_bounds__(256) merge_kernel(const __grid_constant__ PagedParams p)
{
    cudaGridDependencySynchronize();  // the blocks' partials
    const int4 info = p.info[blockIdx.x];
    const int k = info.z + 1;
    if (info.z <= 0)
        return;
    const int32_t h = ROWS == kPagedRows ? info.y : info.y / p.row_groups;
    const int32_t r0 = ROWS == kPagedRows ? 0 : (info.y - h * p.row_groups) * ROWS;
    const int own = 2 * blockIdx.x, step = 2 * (ROWS == kPagedRows ? 1 : p.row_groups);
    auto slot = [&](int i) { return i == 0 ? own + 1 : own + i * step; };
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // row r of the group -> output row, or -1
    auto target = [&](int r) -> int64_t {
        const int32_t rr = r0 + r;
        int32_t gh, tq;
        split_row(p, rr, gh, tq);
        if (rr >= p.G * p.T || tq >= info.w)
            return -1;
        return ((int64_t)info.x * p.Hq + h * p.G + gh) * p.T + tq;
    };
    constexpr int kPerRow = D / 4;  // lanes of 4 features
    if constexpr (!BLOCK_A_ROW) {
        constexpr int kGroups = 32 / kPerRow;
        const int grp = lane / kPerRow, f = lane % kPerRow;
        for (int r = warp; r < ROWS; r += 8) {
            const int64_t at = target(r);
            if (at < 0)
                continue;
            float4 y[16 / kGroups];  // of 16 partials, all on their way at once
            auto fetch = [&](int c) {
#pragma unroll
                for (int i = 0; i < 16; i += kGroups)
                    if (c + i + grp < k)
                        y[i / kGroups] = *reinterpret_cast<const float4*>(
                            p.part_o + (slot(c + i + grp) * ROWS + r) * D + f * 4);
            };
            auto references = [&](int i) {
                return i < k ? p.part_ndl[slot(i) * ROWS + r]
                             : make_float4(kNone, 0.f, 0.f, 0.f);
            };
            auto warp_max = [](float x) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1)
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
                return x;
            };
            fetch(0);
            float4 ndl = references(lane);
            float nx = ndl.x, dx = 0.f;
            bool apart = ndl.y != 0.f;
            for (int i = lane + 32; i < k; i += 32) {
                const float4 more = references(i);
                nx = fmaxf(nx, more.x);
                apart |= more.y != 0.f;
            }
            nx = warp_max(nx);
            if (F8 && __any_sync(0xffffffffu, apart)) {
                dx = (ndl.x - nx) + ndl.y;
                for (int i = lane + 32; i < k; i += 32) {
                    const float4 more = references(i);
                    dx = fmaxf(dx, (more.x - nx) + more.y);
                }
                dx = warp_max(dx);
            }
            float L = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int c = 0;;) {
                const float w = ex2((ndl.x - nx) + (ndl.y - dx));
                if (lane < 16)
                    L += ndl.z * ex2(ndl.x - nx);
#pragma unroll
                for (int i = 0; i < 16; i += kGroups) {
                    const float wi = __shfl_sync(0xffffffffu, w, i + grp);
                    if (c + i + grp < k) {
                        const float4 x = y[i / kGroups];
                        o.x = fmaf(wi, x.x, o.x), o.y = fmaf(wi, x.y, o.y);
                        o.z = fmaf(wi, x.z, o.z), o.w = fmaf(wi, x.w, o.w);
                    }
                }
                c += 16;
                if (c >= k)
                    break;
                fetch(c);
                ndl = references(c + (lane & 15));
            }
#pragma unroll
            for (int i = 8; i > 0; i >>= 1)
                L += __shfl_xor_sync(0xffffffffu, L, i, 16);
            L = __shfl_sync(0xffffffffu, L, 0);
            if (kGroups == 2) {
                o.x += __shfl_xor_sync(0xffffffffu, o.x, 16);
                o.y += __shfl_xor_sync(0xffffffffu, o.y, 16);
                o.z += __shfl_xor_sync(0xffffffffu, o.z, 16);
                o.w += __shfl_xor_sync(0xffffffffu, o.w, 16);
            }
            if (grp == 0)
                write_row<D, F8>(p, at, f * 4, nx, dx, L, o);
        }
    } else {
        constexpr int kGroups = 256 / kPerRow, kAhead = 4;
        __shared__ float wt[kPagedMaxCtas], red_n[8], red_d[8], red_l[8];
        __shared__ float4 acc[256];
        const int grp = threadIdx.x / kPerRow, f = threadIdx.x % kPerRow;
        const int r = blockIdx.y;
        const int64_t at = target(r);
        if (at < 0)
            return;
        auto partial = [&](int i) {
            return *reinterpret_cast<const float4*>(p.part_o + (slot(i) * ROWS + r) * D + f * 4);
        };
        float4 y[kAhead];  // on their way while the weights are made
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (grp + i * kGroups < k)
                y[i] = partial(grp + i * kGroups);
        auto block_max = [&](float x, float(&red)[8]) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
            if (lane == 0)
                red[warp] = x;
            __syncthreads();
            for (int w = 0; w < 8; ++w)
                x = fmaxf(x, red[w]);
            return x;
        };
        float4 ndl[kPagedMaxCtas / 256];
        float nx = kNone, dx = -INFINITY;
#pragma unroll
        for (int i = 0; i < kPagedMaxCtas / 256; ++i) {
            const int at_i = threadIdx.x + i * 256;
            ndl[i] = at_i < k ? p.part_ndl[slot(at_i) * ROWS + r]
                              : make_float4(kNone, 0.f, 0.f, 0.f);
            nx = fmaxf(nx, ndl[i].x);
        }
        nx = block_max(nx, red_n);
        if (F8) {
#pragma unroll
            for (int i = 0; i < kPagedMaxCtas / 256; ++i)
                dx = fmaxf(dx, (ndl[i].x - nx) + ndl[i].y);
            dx = block_max(dx, red_d);
        } else {
            dx = 0.f;
        }
        float L = 0.f;
#pragma unroll
        for (int i = 0; i < kPagedMaxCtas / 256; ++i) {
            wt[threadIdx.x + i * 256] = ex2((ndl[i].x - nx) + (ndl[i].y - dx));
            L += ndl[i].z * ex2(ndl[i].x - nx);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            L += __shfl_xor_sync(0xffffffffu, L, o);
        if (lane == 0)
            red_l[warp] = L;
        __syncthreads();
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        auto add = [&](float w, const float4& x) {
            o.x = fmaf(w, x.x, o.x), o.y = fmaf(w, x.y, o.y);
            o.z = fmaf(w, x.z, o.z), o.w = fmaf(w, x.w, o.w);
        };
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (grp + i * kGroups < k)
                add(wt[grp + i * kGroups], y[i]);
#pragma unroll 4
        for (int i = grp + kAhead * kGroups; i < k; i += kGroups)
            add(wt[i], partial(i));
        acc[threadIdx.x] = o;
        __syncthreads();
        if (grp == 0) {
            L = 0.f;
            for (int w = 0; w < 8; ++w)
                L += red_l[w];
            for (int i = 1; i < kGroups; ++i) {
                const float4 x = acc[i * kPerRow + f];
                o.x += x.x, o.y += x.y, o.z += x.z, o.w += x.w;
            }
            write_row<D, F8>(p, at, f * 4, nx, dx, L, o);
        }
    }
}

template <int D, bool F8, int NB, bool TWO_TERMS>
cudaError_t launch(const CUtensorMap& tk, const CUtensorMap& tv, PagedParams& p,
                   int num_sms, cudaStream_t stream)
{
    using C = Cfg<D, F8, NB>;
    cudaError_t e = cudaFuncSetAttribute(decode_kernel<D, F8, NB, TWO_TERMS>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess)
        return e;
    // as many blocks as are resident at once, no more than there can be pieces
    const int64_t segments = (int64_t)p.c.B * p.c.Hkv;  // of one row group
    const int32_t longest = max(1, ceil_div(p.c.max_pages * p.c.page, kTile));
    p.whole = longest <= kWhole;
    const int64_t pieces = min(segments, (int64_t)kPagedMaxCtas) * (p.whole ? 1 : longest);
    const int resident = min(kPagedMaxCtas, C::kResident * num_sms);
    p.line_blocks = (int)min((int64_t)max(1, resident / p.row_groups), pieces);
    const int grid = p.line_blocks * p.row_groups;
    p.segment_cost = C::kSegmentCost;
    // A grid of at most one block an SM may be launched while the kernel before it ends
    // (its blocks wait at their beginning): one sequence of 1000 rows, called one after
    // the other, 12.3 -> 11.1 us, bf16 with 16 rows 14.4 -> 11.9.  A larger one starts
    // on empty SMs: its blocks are as many as fit, and where a kernel before it still
    // held some SMs they would be dealt out unevenly; 64 ragged sequences then took 104 us
    // instead of 91.
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = grid <= num_sms ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, decode_kernel<D, F8, NB, TWO_TERMS>, tk, tv, p);
    if (e != cudaSuccess || p.whole)
        return e;
    // The merge's blocks may start while the decode's end, and wait there.  With so few
    // segments that each is cut into more partials than a warp takes at once, a block
    // a row.  Measured (8 bits, 8K rows; a block a row, a warp a row): 2, 3, 5 sequences of 8
    // heads 13.1 14.4, 14.9 15.5, 18.4 18.2 us; one of 1 head 13.5 22.1 (20K rows).
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = 1;
    const bool block_a_row = segments * 15 < p.line_blocks;
    cfg.gridDim = dim3(grid, block_a_row ? C::kRows : 1);
    cfg.blockDim = dim3(256);
    return cudaLaunchKernelEx(&cfg, block_a_row ? merge_kernel<D, F8, C::kRows, true>
                                                : merge_kernel<D, F8, C::kRows, false>, p);
}

template <int D, bool F8>
cudaError_t launch_rows(const CUtensorMap& tk, const CUtensorMap& tv, PagedParams& p,
                        int num_sms, cudaStream_t stream)
{
    if (p.G * p.T <= kPagedRows)
        return launch<D, F8, 1, true>(tk, tv, p, num_sms, stream);
    if (F8 && !p.o_fp32)  // (see "Rounding" above)
        return launch<D, F8, 2, !F8>(tk, tv, p, num_sms, stream);
    return launch<D, F8, 2, true>(tk, tv, p, num_sms, stream);
}

}  // namespace paged

cudaError_t launch_decode_paged(const CUtensorMap& tk, const CUtensorMap& tv,
                                PagedParams& p, int num_sms, cudaStream_t stream)
{
    if (p.c.e4m3)
        return p.c.d == 128 ? paged::launch_rows<128, true>(tk, tv, p, num_sms, stream)
                            : paged::launch_rows<64, true>(tk, tv, p, num_sms, stream);
    return p.c.d == 128 ? paged::launch_rows<128, false>(tk, tv, p, num_sms, stream)
                        : paged::launch_rows<64, false>(tk, tv, p, num_sms, stream);
}

}  // namespace dfa
