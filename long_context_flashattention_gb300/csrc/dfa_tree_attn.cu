// dfa_tree_attn.cu -- attention of trees of drafted tokens over a paged key/value cache, on
// the tensor cores: the nodes of a tree, times the query heads that share a key/value
// head, against the rows of their sequence.
//
// Method.  With keys k_j = s_j c_j and values v_j = u_j w_j (codes and scales; 1 for bf16
// cells), a query row has x_j = scale log2(e) s_j (q . c_j) and
//   O = 2^D (sum_j 2^(x_j - N + log2 u_j - D) w_j) / (sum_j 2^(x_j - N)),
//   LSE = ln 2 (N + log2 sum),
// with N the running maximum of the scores, and D that of the weights' exponents beyond it
// (0 for bf16 cells), so that weights fit their type whatever the scales are.  A score is
// rounded to fp32 before N is taken off it, as N was when it was one of them: the
// difference is exact however large both are.  Weights are the sum's terms times
// 2^(log2 u_j - D), where every u_j of a tile is in [2^-40, 2^40], and else powers of their
// own.
//
// What a node sees: every row before the tree, and of the tree's rows those whose bits
// its mask has.  Only tiles that reach into the tree or over the sequence's end look at
// masks; a row of the tile is 128 bits.
//
// A block (one an SM) keeps 128 query rows (TILES = 1), or 256 (TILES = 2), and walks over
// 128-key tiles of the cache:
//   warp 9       pages by TMA into a ring of K and V tiles, 128-byte swizzle;
//   warps 12-15  (8-bit cells) those to fp16, in the same layout;
//   warps 10-11  a segment's queries (8-bit cells: fp16 relative to a power of two of the
//                row: exact but for elements below 2^-31 of its largest one);
//   warp 8       S = Q K^T into TMEM, O += P V with P from TMEM (over S's columns);
//   warps 0-7    softmax, a thread a row, O rescaled in TMEM when M has to rise.  TILES =
//                1: the two groups of four warps take the tiles in turn, each with an O, M
//                and sum of its own, joined at the segment's end; TILES = 2: 128 rows each.
//
// Work: (sequence, head, row group) segments form one line, cut by cost over a grid of
// one block an SM: a block's range covers whole segments, whose result it writes, and up
// to two cut ones, whose partials merge_kernel joins.  The lengths are read on the
// device, so a captured graph follows them.
//
// Rounding: weights as two bf16 terms (2^-16) for bf16 cells; for 8-bit cells as one fp16
// term (2^-11) with a bf16 output, as two (2^-22) with an fp32 one.  Sums, maxima and O in
// fp32.
//
// Values that are not finite, in a row that some nodes see and others do not, would reach
// the others as 0 * inf.  Such rows (looked for in tiles that reach into the tree) are
// taken out of the products, and the nodes that see them add them at the segment's end.
#include <cfloat>

#include "dfa_branch.h"
#include "dfa_serve.cuh"

namespace dfa {

namespace tree {

constexpr int kTile = kTreeTile;
constexpr int kRing = 8;                  // tiles whose scales are kept
constexpr int kRuns = 4;                  // segments that are announced ahead
constexpr float kGrow = 8.f;              // N rises when a term exceeds 2^8
// D is set kHead below the largest exponent, and set anew when a weight exceeds 2^kTop
// (fp16 weights use that type's range to its end, so that those far below the largest
// keep their bits).
constexpr float kTop = 15.f, kHead = 11.f;
constexpr float kNone = -FLT_MAX;         // running maximum before the first key
constexpr float kNear = 40.f;             // terms times 2^(log2 u_j - D) are weights while
                                          // |log2 u_j| is at most this
constexpr float kLn2 = 0.69314718055994531f;
// Where no sequence can be longer than so many tiles, segments are not cut and there is
// nothing to merge.
constexpr int kWhole = 2;
constexpr uint32_t kWideTile = 256;       // flag of a tile, beside the missing pages' bits

// A run of tiles [tile0, tile0 + nt) of one segment: key/value head h, row group rg of
// sequence b, which has len rows, n nodes and that many tiles.
struct Piece {
    int32_t b, h, rg, len, n;
    int32_t tile0, nt, tiles;
    long long w;  // the segment's first unit on the line
};

template <int D, bool F8, int TILES>
struct Cfg {
    static constexpr int kThreads = F8 ? 512 : 384;
    static constexpr int kRows = TILES * kTreeRows;
    static constexpr int kTileBytes = kTile * D * 2;      // a K, V or Q tile of 16-bit elements
    static constexpr int kRawBytes = kTile * D;
    static constexpr int kSlots = F8 ? (D == 128 ? 3 : 4) : (D == 128 ? 5 : 8);
    static constexpr int kRaw = !F8 ? 0 : D == 128 ? (TILES == 1 ? 5 : 3) : 6;
    static constexpr int kQ0 = 0;
    static constexpr int kSlot0 = TILES * kTileBytes;
    static constexpr int kRaw0 = kSlot0 + kSlots * kTileBytes;
    static constexpr int kShared0 = kRaw0 + kRaw * kRawBytes;
    static constexpr int kCopies = F8 ? kRaw : kSlots;    // slots that TMA fills
    // Registers: the threads' total at launch is shared out anew.
    static constexpr int kRegsMath = 192;
    static constexpr int kRegsCtl = F8 ? 56 : 120;
    static constexpr int kRegsConv = 72;
    static_assert(F8 ? 2 * kRegsMath + kRegsCtl + kRegsConv == 4 * 128
                     : 2 * kRegsMath + kRegsCtl == 3 * 168, "register budget");
    static constexpr int kReaders = 8 + 1 + 2 + (F8 ? 4 : 0);  // warps that read a run
};

struct TileInfo {
    float2 scale[8];   // per page: K's scale, log2 of V's
    uint32_t flags;    // pages that are not there; kWideTile
    uint32_t pad;
};

template <int D, bool F8, int TILES>
struct Shared {
    using C = Cfg<D, F8, TILES>;
    uint64_t full[C::kSlots], empty[C::kSlots];           // tiles for the products
    uint64_t raw_full[F8 ? C::kRaw : 1], raw_empty[F8 ? C::kRaw : 1];
    uint64_t s_full[2], p_full[2], o_full, o_empty, q_full, q_empty;
    uint64_t run_full[kRuns], run_empty[kRuns], info_full[kRing], meet;
    Piece run[kRuns];
    TileInfo info[kRing];
    long long warp_sum[16];
    long long w0, w1, base, each, rest;
    int32_t b, block;
    uint32_t tmem, abort;
    uint32_t bad[3][32];       // nodes whose values are not finite
    uint32_t any_bad[3];
    float qf[F8 ? C::kRows : 1];                          // score factors of the rows
    // of the two groups, where they share the rows: N, D, sum; two sets, since a group
    // may end the next segment while the other still reads this one's
    static constexpr int kBoth = TILES == 1 ? kTreeRows : 1;
    float n[2][2][kBoth], l[2][2][kBoth], d[2][2][F8 ? kBoth : 1];
};

template <int D, bool F8, int TILES>
constexpr int kSmem = Cfg<D, F8, TILES>::kShared0 + (int)sizeof(Shared<D, F8, TILES>) + 1024;

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

__device__ __forceinline__ void mbar_expect(uint64_t* bar, uint32_t bytes)
{
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)),
                 "r"(bytes)
                 : "memory");
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

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Instruction descriptor with fp16 or bf16 operands.
template <bool F16>
constexpr uint32_t idesc(int N, bool b_mn_major)
{
    return F16 ? idesc_bf16_f32(128, N, false, b_mn_major) & ~((1u << 7) | (1u << 10))
               : idesc_bf16_f32(128, N, false, b_mn_major);
}

// Query row r of a key/value head: head of the group and node.
__device__ __forceinline__ void split_row(const TreeParams& p, int32_t r, int32_t& gh, int32_t& tq)
{
    gh = (int32_t)(((uint32_t)r * p.inv_T) >> 21);  // r / T: r below 2^11
    tq = r - gh * p.T;
}

// Tiles of a sequence with n nodes: at least one, so that rows without keys are
// written too.
__device__ __forceinline__ int32_t tiles_of(int32_t len, int32_t n)
{
    return n > 0 ? max(1, ceil_div(len, kTile)) : 0;
}

// a / b for a >= 0, b > 0, the short way where a has 32 bits
__device__ __forceinline__ long long divide(long long a, int32_t b)
{
    return a >> 32 ? a / b : (long long)((uint32_t)a / (uint32_t)b);
}

// The line that is cut: every segment takes p.segment_cost units (its queries, the join
// and the rows' output cost a block about that many tiles' time), then one unit per
// tile.  A cut inside the former puts the whole segment behind it.
//
// One warp's way along the block's range.  (Lengths that change while the kernel runs
// give results without meaning, but nothing worse: only this warp goes by them, and
// every index that comes of them is checked.)
struct Walk : Piece {
    long long w1;  // end of the range
    bool fresh;    // tile0 is where the range begins

    template <typename SH>
    __device__ __forceinline__ void start(const TreeParams& p, const SH& sh, int32_t group)
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
    __device__ __forceinline__ bool next(const TreeParams& p)
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

// The block's range of the line, and the sequence that it begins in.
template <int THREADS, typename SH>
__device__ __forceinline__ void find_range(const TreeParams& p, SH& sh)
{
    const int32_t per_seq = p.c.Hkv;
    const int32_t chunk = ceil_div(p.c.B, THREADS);
    const int32_t block = blockIdx.x / p.row_groups;
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
    for (int w = 0; w < THREADS / 32; ++w) {
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

// The block of the group whose range has this unit.
template <typename SH>
__device__ __forceinline__ int block_of(const TreeParams& p, const SH& sh, long long unit)
{
    const long long longer = sh.rest * (sh.each + 1);
    const long long c = unit < longer ? unit / (sh.each + 1) : sh.rest + (unit - longer) / sh.each;
    return (int)min(c, (long long)p.line_blocks - 1);
}

// The next segment that the producer announced, in every lane; false: no more, or the
// block is giving up.
template <typename SH>
__device__ __forceinline__ bool next_run(SH& sh, uint32_t seg, Piece& run, const WaitCtx& wctx,
                                         int where)
{
    const bool ok = mbar_wait(&sh.run_full[seg % kRuns], (seg / kRuns) & 1, wctx, where);
    if (!__all_sync(0xffffffffu, ok))
        return false;
    run = sh.run[seg % kRuns];
    __syncwarp();
    if ((threadIdx.x & 31) == 0)
        mbar_arrive(&sh.run_empty[seg % kRuns]);
    return run.nt > 0;
}

// ---------------------------------------------------------------------------
// producer: the tiles' pages, and what there is to know of them
// ---------------------------------------------------------------------------
template <int D, bool F8, int TILES>
__device__ __forceinline__ void produce(const TreeParams& p, Shared<D, F8, TILES>& sh,
                                        uint32_t slots, const CUtensorMap& tk,
                                        const CUtensorMap& tv, const WaitCtx& wctx)
{
    using C = Cfg<D, F8, TILES>;
    constexpr int kPlanes = F8 ? 1 : D / 64;            // boxes side by side
    constexpr int kBoxRow = F8 ? D : 128;               // bytes of a box's row
    constexpr int kBytes = F8 ? C::kRawBytes : C::kTileBytes;
    const int lane = threadIdx.x & 31;
    const int32_t page = p.c.page;
    const int32_t per_tile = kTile / page;
    uint64_t* full = F8 ? sh.raw_full : sh.full;
    uint64_t* empty = F8 ? sh.raw_empty : sh.empty;
    uint32_t st = 0, phase = 0, seg = 0, gt = 0;
    Walk wk;
    wk.start(p, sh, blockIdx.x - sh.block * p.row_groups);
    bool more = wk.next(p);
    // Table entry of this lane's page of the 32 from page `win` on; -1: none.
    auto entry = [&](const Walk& x, int32_t win) {
        const int32_t end = ceil_div(min(x.len, (x.tile0 + x.nt) * kTile), page);
        return win + lane < end ? page_entry(p.c, x.b, win + lane) : -1;
    };
    auto announce = [&](bool end) {
        const bool ok = mbar_wait(&sh.run_empty[seg % kRuns], (seg / kRuns + 1) & 1, wctx, 51);
        if (!__all_sync(0xffffffffu, ok))
            return false;
        if (lane == 0) {
            sh.run[seg % kRuns] = wk;
            if (end)
                sh.run[seg % kRuns].nt = 0;
            mbar_arrive(&sh.run_full[seg % kRuns]);
        }
        return true;
    };
    int32_t next_id = more ? entry(wk, (wk.tile0 * kTile) >> p.c.page_log2) : -1;
    for (; more; ++seg) {
        if (!announce(false))
            return;
        const int32_t h = wk.h;
        const int32_t pages_end = ceil_div(min(wk.len, (wk.tile0 + wk.nt) * kTile), page);
        int32_t win = (wk.tile0 * kTile) >> p.c.page_log2, id = next_id;
        float ks = 1.f, vs = 1.f;
        auto check_window = [&] {  // the lane's page, and its scales on their way
            if (win + lane >= pages_end || !is_page(p.c, wk.b, id)) {
                id = -1;
            } else if (F8) {
                const int64_t at = (int64_t)id * p.c.Hkv + h;
                ks = __ldcg(p.c.k_scale + at);
                vs = __ldcg(p.c.v_scale + at);
            }
        };
        check_window();
        Walk nx = wk;
        bool more_next = false;
        const int32_t look = min(wk.nt - 1, 2);
        for (int32_t i = 0; i < wk.nt; ++i, ++gt) {
            const int32_t key0 = (wk.tile0 + i) * kTile;
            const int32_t p0 = key0 >> p.c.page_log2;
            if (p0 >= win + 32) {
                win = p0;
                id = entry(wk, win);
                check_window();
            }
            const int src = p0 - win + lane;  // lanes below per_tile: their box's page
            const int32_t my = __shfl_sync(0xffffffffu, id, src & 31);
            const bool load = lane < per_tile && p0 + lane < pages_end && my >= 0;
            const uint32_t boxes = __ballot_sync(0xffffffffu, load);
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                // (passes at once in the first round: the phase before the barrier's first)
                const bool ok = mbar_wait(&empty[st], phase ^ 1, wctx, 50);
                if (!__all_sync(0xffffffffu, ok))
                    return;
                if (lane == 0)
                    mbar_expect(&full[st], __popc(boxes) * (page * D * (F8 ? 1 : 2)));
                __syncwarp();
                if (load) {
                    const uint32_t dst = slots + st * kBytes + lane * page * kBoxRow;
#pragma unroll
                    for (int pl = 0; pl < kPlanes; ++pl)
                        tma_load_4d(dst + pl * kTile * 128, kv ? &tv : &tk, &full[st], pl * 64, 0,
                                    h, my);
                }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&full[st]);
                if (++st == C::kCopies) {
                    st = 0;
                    phase ^= 1;
                }
            }
            // What the softmax has to know.  (A tile's entry is written anew kRing tiles
            // later, when the ring's slots say that its softmax is long done.)
            TileInfo& info = sh.info[gt % kRing];
            const float my_ks = __shfl_sync(0xffffffffu, ks, src & 31);
            const float my_vs = __shfl_sync(0xffffffffu, vs, src & 31);
            float lu = 0.f;
            if (F8 && load) {
                // exponent and significand apart: exact for a power of two
                const uint32_t bits = __float_as_uint(my_vs);
                const int e = (int)((bits >> 23) & 0xffu);
                lu = e == 255 ? my_vs : (float)max(e - 127, -126) +
                                            log2f(__uint_as_float((bits & 0x7fffffu) | (127u << 23)));
            }
            const bool wide = F8 && __any_sync(0xffffffffu, !(fabsf(lu) <= kNear));
            if (lane < per_tile)
                info.scale[lane] = make_float2(load ? my_ks : 0.f, lu);
            const uint32_t missing = ~boxes & ((1u << per_tile) - 1);
            if (lane == 0)
                info.flags = missing | (wide ? kWideTile : 0u);
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sh.info_full[gt % kRing]);
            if (i == look) {
                more_next = nx.next(p);
                next_id = more_next ? entry(nx, (nx.tile0 * kTile) >> p.c.page_log2) : -1;
            }
        }
        wk = nx;
        more = more_next;
    }
    announce(true);
}

// ---------------------------------------------------------------------------
// queries of the segments
// ---------------------------------------------------------------------------
template <int D, bool F8, int TILES>
__device__ __forceinline__ void load_queries(const TreeParams& p, Shared<D, F8, TILES>& sh,
                                             uint32_t qs, const WaitCtx& wctx)
{
    using C = Cfg<D, F8, TILES>;
    constexpr int kPerRow = D / 8;                 // lanes of a row, 8 elements each
    constexpr int kRowsAt = 64 / kPerRow;          // rows of the two warps at a time
    constexpr int kBatch = 4;
    const int t = threadIdx.x & 63, c = t % kPerRow;
    Piece run;
    for (uint32_t seg = 0; next_run(sh, seg, run, wctx, 53); ++seg) {
        const bool ok = mbar_wait(&sh.q_empty, (seg & 1) ^ 1, wctx, 54);
        if (!__all_sync(0xffffffffu, ok))
            return;
        for (int32_t r0 = t / kPerRow; r0 < C::kRows; r0 += kBatch * kRowsAt) {
            uint4 x[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int32_t r = run.rg * C::kRows + r0 + k * kRowsAt;
                int32_t gh, tq;
                split_row(p, r, gh, tq);
                x[k] = make_uint4(0, 0, 0, 0);
                if (r < p.G * p.T && tq < run.n)
                    x[k] = *reinterpret_cast<const uint4*>(
                        (const __nv_bfloat16*)p.q.p + run.b * p.q.sb +
                        (int64_t)(run.h * p.G + gh) * p.q.sh + (int64_t)tq * p.q.sl + c * 8);
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int32_t row = r0 + k * kRowsAt;
                if (F8) {
                    uint32_t* w = &x[k].x;
                    float amax = 0.f;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        amax = fmaxf(amax, fmaxf(fabsf(bf16lo(w[i])), fabsf(bf16hi(w[i]))));
#pragma unroll
                    for (int o = 1; o < kPerRow; o <<= 1)
                        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                    // the largest element to [2^14, 2^15): those down to 2^-31 of it stay exact
                    const int e = min(max((int)(__float_as_uint(amax) >> 23) - 127, -100), 126) - 14;
                    const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        w[i] = pack_half2(bf16lo(w[i]) * inv, bf16hi(w[i]) * inv);
                    if (c == 0)
                        sh.qf[row] = p.scale_log2 * __uint_as_float((uint32_t)(127 + e) << 23);
                }
                st_shared_v4(qs + (row / kTreeRows) * C::kTileBytes + (c >> 3) * (kTreeRows * 128) +
                                 sw128_offset(row % kTreeRows, c & 7),
                             x[k].x, x[k].y, x[k].z, x[k].w);
            }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if ((t & 31) == 0)
            mbar_arrive(&sh.q_full);
    }
}

// ---------------------------------------------------------------------------
// 8-bit cells to fp16
// ---------------------------------------------------------------------------
// A warp takes 32 rows.  Eight lanes at a time read 16 bytes each and write twice that,
// which the swizzles keep free of bank conflicts where the two rows they are of differ in
// bits 0 and 2 (128-byte rows), or in bit 0 (64-byte rows, two to a line).
template <int D, int TILES>
__device__ __forceinline__ void convert(const TreeParams& p, Shared<D, true, TILES>& sh,
                                        uint32_t slots, uint32_t raw, const WaitCtx& wctx)
{
    using C = Cfg<D, true, TILES>;
    const int warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
    const int sub = lane & 7, g = lane >> 3;
    uint32_t rs = 0, rphase = 0, st = 0, phase = 0;
    Piece run;
    for (uint32_t seg = 0; next_run(sh, seg, run, wctx, 55); ++seg) {
        for (int32_t i = 0; i < 2 * run.nt; ++i) {
            bool ok = mbar_wait(&sh.raw_full[rs], rphase, wctx, 56);
            ok = ok && mbar_wait(&sh.empty[st], phase ^ 1, wctx, 57);
            if (!__all_sync(0xffffffffu, ok))
                return;
            const uint32_t from = raw + rs * C::kRawBytes, to = slots + st * C::kTileBytes;
#pragma unroll
            for (int it = 0; it < D / 16; ++it) {
                uint32_t row, ch, src;
                if (D == 128) {
                    row = warp * 32 + (it >> 1) * 8 + ((sub >> 2) ? g ^ 5 : g);
                    ch = (sub & 3) + 4 * (it & 1);
                    src = row * 128 + ((ch ^ (row & 7)) << 4);
                } else {
                    row = warp * 32 + it * 8 + g * 2 + (sub >> 2);
                    ch = sub & 3;
                    src = row * 64 + ((ch ^ ((row >> 1) & 3)) << 4);
                }
                const uint4 x = lds128(from + src);
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t c16 = 2 * ch + e;
                    st_shared_v4(to + (c16 >> 3) * (kTile * 128) + sw128_offset(row, c16 & 7),
                                 e4m3x2_half2(w[2 * e] & 0xffffu), e4m3x2_half2(w[2 * e] >> 16),
                                 e4m3x2_half2(w[2 * e + 1] & 0xffffu),
                                 e4m3x2_half2(w[2 * e + 1] >> 16));
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sh.full[st]);
                mbar_arrive(&sh.raw_empty[rs]);
            }
            if (++rs == C::kRaw) {
                rs = 0;
                rphase ^= 1;
            }
            if (++st == C::kSlots) {
                st = 0;
                phase ^= 1;
            }
        }
    }
}

// ---------------------------------------------------------------------------
// products, issued by one thread
// ---------------------------------------------------------------------------
template <int D, bool F8, int TILES, bool TWO>
__device__ __forceinline__ void multiply(Shared<D, F8, TILES>& sh, uint32_t qs, uint32_t slots,
                                         uint32_t tmem, const WaitCtx& wctx)
{
    using C = Cfg<D, F8, TILES>;
    const int lane = threadIdx.x & 31;
    const uint64_t dQ = sdesc_sw128(qs, 16, 1024);
    const uint64_t dK = sdesc_sw128(slots, 16, 1024);
    const uint64_t dV = sdesc_sw128(slots, 16384, 1024);
    uint32_t gt = 0;
    // slot and phase of the next K tile, and of the V tile whose product is next
    uint32_t ks = 0, kphase = 0, vs = 1, vphase = 0;
    auto two_on = [](uint32_t& s, uint32_t& ph) {
        s += 2;
        if (s >= (uint32_t)C::kSlots) {
            s -= C::kSlots;
            ph ^= 1;
        }
    };
    auto scores = [&](int t, int w) {  // S_w = Q_t K^T
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
            mma_ss(tmem + w * 128, sdesc_add(dQ, t * C::kTileBytes + off),
                   sdesc_add(dK, ks * C::kTileBytes + off), idesc<F8>(128, false), kk > 0);
        }
        tc_commit(&sh.s_full[w]);
    };
    auto outputs = [&](int w, bool add) {  // O_w += P_w V
#pragma unroll
        for (int kk = 0; kk < (TWO ? 16 : 8); ++kk)
            mma_ts(tmem + 256 + w * D, tmem + w * 128 + kk * 8,
                   sdesc_add(dV, vs * C::kTileBytes + (kk & 7) * 2048), idesc<F8>(D, true),
                   (add || kk > 0) ? 1u : 0u);
    };
    uint32_t pc[2] = {0, 0};
    Piece run;
    for (uint32_t seg = 0; next_run(sh, seg, run, wctx, 20); ++seg) {
        bool ok = true;
        if (lane == 0) {
            const int32_t nt = run.nt;
            ok = mbar_wait(&sh.q_full, seg & 1, wctx, 21);
            auto next_scores = [&](bool last) {
                ok = ok && mbar_wait(&sh.full[ks], kphase, wctx, 22);
                if (!ok)
                    return;
                tc_fence_after();
                scores(0, gt & 1);
                tc_commit(&sh.empty[ks]);
                if (last)
                    tc_commit(&sh.q_empty);
                two_on(ks, kphase);
            };
            if (TILES == 1) {
                // gt counts the tiles whose scores are next
                if (ok)
                    next_scores(nt == 1);
                ++gt;
                for (int32_t i = 0; ok && i < nt; ++i) {
                    if (i + 1 < nt) {
                        next_scores(i + 2 == nt);
                        ++gt;
                    }
                    const uint32_t w = (gt - (i + 1 < nt ? 2 : 1)) & 1;
                    ok = ok && (i > 0 || mbar_wait(&sh.o_empty, (seg & 1) ^ 1, wctx, 23)) &&
                         mbar_wait(&sh.full[vs], vphase, wctx, 24) &&
                         mbar_wait(&sh.p_full[w], pc[w] & 1, wctx, 25);
                    if (!ok)
                        break;
                    ++pc[w];
                    tc_fence_after();
                    outputs(w, i >= 2);
                    tc_commit(&sh.empty[vs]);
                    two_on(vs, vphase);
                }
            } else {
                for (int32_t i = -1; ok && i < nt; ++i) {
                    if (i >= 0)
                        ok = ok && (i > 0 || mbar_wait(&sh.o_empty, (seg & 1) ^ 1, wctx, 23)) &&
                             mbar_wait(&sh.full[vs], vphase, wctx, 24);
                    if (i + 1 < nt)
                        ok = ok && (i >= 0 || mbar_wait(&sh.full[ks], kphase, wctx, 22));
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        if (i >= 0) {
                            ok = ok && mbar_wait(&sh.p_full[w], pc[w] & 1, wctx, 25 + w);
                            ++pc[w];
                            tc_fence_after();
                            if (ok)
                                outputs(w, i > 0);
                            if (w == 1 && ok)
                                tc_commit(&sh.empty[vs]);
                            if (w == 0 && i + 1 < nt)
                                ok = ok && mbar_wait(&sh.full[ks], kphase, wctx, 22);
                        }
                        if (i + 1 < nt && ok) {
                            tc_fence_after();
                            scores(w, w);
                            if (w == 1) {
                                tc_commit(&sh.empty[ks]);
                                if (i + 2 == nt)
                                    tc_commit(&sh.q_empty);
                            }
                        }
                    }
                    if (i >= 0)
                        two_on(vs, vphase);
                    if (i + 1 < nt)
                        two_on(ks, kphase);
                }
            }
            if (ok)
                tc_commit(&sh.o_full);
        }
        if (!__shfl_sync(0xffffffffu, (int)ok, 0))
            return;
    }
}

// ---------------------------------------------------------------------------
// softmax
// ---------------------------------------------------------------------------
// Which of the 128 keys from key `base` on a node sees: of the rows before the tree all,
// of the tree's those of its mask (NULL: none), of missing pages none.
__device__ __forceinline__ void visible(const TreeParams& p, const Piece& run, int32_t base,
                                        const uint32_t* mask, uint32_t missing, uint32_t (&vis)[4])
{
    const int32_t tree0 = run.len - run.n;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int32_t k0 = base + 32 * i, off = k0 - tree0;  // node of the word's first key
        uint32_t bits = off <= -32 ? ~0u : off < 0 ? (1u << -off) - 1 : 0u;
        if (mask && off > -32 && off < run.n) {
            uint32_t m;
            if (off < 0) {
                m = mask[0] << -off;
            } else {
                const int32_t w = off >> 5;
                const uint32_t lo = mask[w], hi = w + 1 < p.words ? mask[w + 1] : 0u;
                m = __funnelshift_r(lo, hi, off & 31);
            }
            const int32_t left = run.n - off;  // nodes from here on
            bits |= left >= 32 ? m : m & ((1u << left) - 1);
        }
        vis[i] = bits;
    }
    if (missing) {
        for (int k = 0; k < kTile / 16; ++k)
            if (missing >> (16 * k >> p.c.page_log2) & 1)
                vis[k >> 1] &= ~(0xffffu << (16 * (k & 1)));
    }
}

// Adds the values of the nodes in `bad`, which the products left out, to features
// [f0, f0 + 32) of a row's O (relative to 2^(N + D)).
template <int D, bool F8>
__device__ __noinline__ void add_apart(const TreeParams& p, const Piece& run, const uint32_t* bad,
                                       const uint32_t* mask, int32_t gh, int32_t tq, float N,
                                       float Dd, int f0, float* o)
{
    const __nv_bfloat16* q = (const __nv_bfloat16*)p.q.p + run.b * p.q.sb +
                             (int64_t)(run.h * p.G + gh) * p.q.sh + (int64_t)tq * p.q.sl;
    for (int32_t u = 0; u < run.n; ++u) {
        if (!(bad[u >> 5] & mask[u >> 5] & (1u << (u & 31))))
            continue;
        const int32_t j = run.len - run.n + u;
        const int32_t id = page_of(p.c, run.b, j >> p.c.page_log2);
        if (id < 0)
            continue;
        const int64_t at = (int64_t)id * p.c.page_stride +
                           (((int64_t)run.h << p.c.page_log2) + (j & (p.c.page - 1))) * D;
        auto cell = [&](const void* cells, int f) {
            return F8 ? e4m3x2_float2(((const uint8_t*)cells)[at + f]).x
                      : __bfloat162float(((const __nv_bfloat16*)cells)[at + f]);
        };
        float dot = 0.f, lu = 0.f;
        for (int f = 0; f < D; ++f)
            dot = fmaf(__bfloat162float(q[f]), cell(p.c.k, f), dot);
        float x = dot * p.scale_log2;
        if (F8) {
            x *= p.c.k_scale[(int64_t)id * p.c.Hkv + run.h];
            lu = log2f(p.c.v_scale[(int64_t)id * p.c.Hkv + run.h]);
        }
        const float w = ex2((x - N) + (lu - Dd));
        for (int f = 0; f < 32; ++f)
            o[f] = fmaf(w, cell(p.c.v, f0 + f), o[f]);
    }
}

// Features f..f+3 of an output row: o is relative to 2^(nx + dx), L to 2^nx.
template <int D, bool F8>
__device__ __forceinline__ float2 row_factors(float dx, float L)
{
    // 2^dx in two halves: it may be below fp32's range where o makes up for it
    const float half = F8 ? ex2(0.5f * dx) : 1.f;
    return make_float2(L == 0.f ? 0.f : half / L, half);  // (NaN stays NaN)
}

__device__ __forceinline__ float row_lse(float nx, float L)
{
    return L == 0.f ? -INFINITY : (nx + log2f(L)) * kLn2;
}

// Zeros rows of a V tile that are not the sequence's or whose page is missing, and rows
// of the tree with values that are not finite, which it notes.  A thread a row.
template <int D, bool F8, typename SH>
__device__ __forceinline__ void mend_values(const TreeParams& p, SH& sh, const Piece& run,
                                            uint32_t vt, int32_t base, int32_t row,
                                            uint32_t missing, uint32_t seg)
{
    const int32_t j = base + row, node = j - (run.len - run.n);
    const bool gone = j >= run.len || (missing >> (row >> p.c.page_log2) & 1);
    if (!gone && node < 0)
        return;
    bool bad = false;
    if (!gone) {
        constexpr uint32_t kHi = F8 ? 0x7c000000u : 0x7f800000u, kLo = F8 ? 0x7c00u : 0x7f80u;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
            const uint4 x = lds128(vt + (c >> 3) * (kTile * 128) + sw128_offset(row, c & 7));
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                bad |= (w[i] & kHi) == kHi || (w[i] & kLo) == kLo;
        }
        if (bad) {
            atomicOr(&sh.bad[seg % 3][node >> 5], 1u << (node & 31));
            sh.any_bad[seg % 3] = 1;
        }
    }
    if (gone || bad) {
#pragma unroll
        for (int c = 0; c < D / 8; ++c)
            st_shared_v4(vt + (c >> 3) * (kTile * 128) + sw128_offset(row, c & 7), 0, 0, 0, 0);
        fence_proxy_async_smem();
    }
}

template <int D, bool F8, int TILES, bool TWO>
__device__ __forceinline__ void softmax(const TreeParams& p, Shared<D, F8, TILES>& sh,
                                        uint32_t slots, uint32_t tmem, const WaitCtx& wctx)
{
    using C = Cfg<D, F8, TILES>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int w = warp >> 2, rit = (warp & 3) * 32 + lane;  // group, row of the tile
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lanes + w * 128, tO = tmem + lanes + 256;
    const int32_t R = p.G * p.T;
    uint32_t gt = 0, sc = 0, met = 0;
    int4 info = make_int4(0, 0, 0, 0);
    Piece run;
    for (uint32_t seg = 0; next_run(sh, seg, run, wctx, 30); ++seg) {
        const int32_t r0 = run.rg * C::kRows + (TILES == 2 ? w * kTreeRows : 0);
        int32_t gh, tq;
        split_row(p, r0 + rit, gh, tq);
        const bool valid = r0 + rit < R && tq < run.n;
        const uint32_t* mask =
            valid ? p.mask + ((int64_t)run.b * p.T + tq) * p.words : nullptr;
        float factor = p.scale_log2;
        if (F8) {
            const bool ok = mbar_wait(&sh.q_full, seg & 1, wctx, 31);
            if (!__all_sync(0xffffffffu, ok))
                return;
            factor = sh.qf[(TILES == 2 ? w * kTreeRows : 0) + rit];
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sh.q_empty);
        }
        float N = kNone, Dd = 0.f, l = 0.f;
        bool first = true;
        for (int32_t i = 0; i < run.nt; ++i, ++gt) {
            if (TILES == 1 && (gt & 1) != (uint32_t)w)
                continue;
            const int32_t base = (run.tile0 + i) * kTile;
            bool ok = mbar_wait(&sh.info_full[gt % kRing], (gt / kRing) & 1, wctx, 32);
            if (!__all_sync(0xffffffffu, ok))
                return;
            const TileInfo& ti = sh.info[gt % kRing];
            const uint32_t flags = ti.flags, missing = flags & 0xffu;
            const bool masked = base + kTile > run.len - run.n || missing;
            uint32_t vis[4];
            if (masked)
                visible(p, run, base, mask, missing, vis);
            ok = mbar_wait(&sh.s_full[w], sc & 1, wctx, 33);
            if (!__all_sync(0xffffffffu, ok))
                return;
            ++sc;
            tc_fence_after();
            uint32_t r[128];
            tmem_ld32(tS + 0, r);
            tmem_ld32(tS + 32, r + 32);
            tmem_ld32(tS + 64, r + 64);
            tmem_ld32(tS + 96, r + 96);
            tmem_ld_wait();
            tmem_reg_fence32(r);
            tmem_reg_fence32(r + 32);
            tmem_reg_fence32(r + 64);
            tmem_reg_fence32(r + 96);
            float x[128];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float fk = F8 ? factor * ti.scale[16 * k >> p.c.page_log2].x : factor;
                const uint64_t f2 = f2pack(fk, fk);
#pragma unroll
                for (int j = 16 * k; j < 16 * k + 16; j += 2)
                    f2unpack(f2mul(f2pack(__uint_as_float(r[j]), __uint_as_float(r[j + 1])), f2),
                             x[j], x[j + 1]);
            }
            if (masked) {
#pragma unroll
                for (int j = 0; j < 128; ++j)
                    x[j] = vis[j / 32] >> (j % 32) & 1 ? x[j] : -INFINITY;
            }
            float top[8];  // of 16 keys each
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                float m = fmaxf(x[16 * k], x[16 * k + 1]);
#pragma unroll
                for (int j = 16 * k + 2; j < 16 * k + 16; j += 2)
                    m = fmax3(m, x[j], x[j + 1]);
                top[k] = m;
            }
            const float mx = fmaxf(fmax3(fmax3(top[0], top[1], top[2]), top[3], top[4]),
                                   fmax3(top[5], top[6], top[7]));
            // N up to the largest score, D up to the largest exponent, O with them
            float f = 1.f;
            bool rise = mx - N > kGrow;
            if (rise) {
                f = ex2(N - mx);
                l *= f;
                Dd += N - mx;
                N = mx;
            }
            if (F8) {
                float me = -INFINITY;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    me = fmaxf(me, (top[k] - N) + ti.scale[16 * k >> p.c.page_log2].y);
                rise = me - Dd > kTop;
                f = 1.f;
                if (rise) {
                    f = ex2(Dd - (me - kHead));
                    Dd = me - kHead;
                }
            }
            // O is as the product of this group's tile before this one left it: it was
            // issued before these scores
            if (!first && __any_sync(0xffffffffu, rise)) {
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 16) {
                    uint32_t o[16];
                    tmem_ld16(tO + w * D + c0, o);
                    tmem_ld_wait();
                    tmem_reg_fence16(o);
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                    tmem_st16(tO + w * D + c0, o);
                }
            }
            first = false;
            const uint64_t off = f2pack(-N, -N);
            const bool wide = F8 && (flags & kWideTile);
            uint64_t sum[2] = {f2pack(0.f, 0.f), f2pack(0.f, 0.f)};
#pragma unroll
            for (int k = 0; k < 4; ++k) {  // 32 keys at a time
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int at = 32 * k + 2 * j;
                    const float lu = F8 ? ti.scale[(at & ~15) >> p.c.page_log2].y - Dd : 0.f;
                    const uint64_t e = f2add(f2pack(x[at], x[at + 1]), off);
                    float a, b;
                    f2unpack(e, a, b);
                    a = ex2(a);
                    b = ex2(b);
                    sum[j & 1] = f2add(sum[j & 1], f2pack(a, b));
                    if (F8) {
                        if (__builtin_expect(wide, 0)) {
                            f2unpack(f2add(e, f2pack(lu, lu)), a, b);
                            a = ex2(a);
                            b = ex2(b);
                        } else {
                            const float g = ex2(lu);
                            f2unpack(f2mul(f2pack(a, b), f2pack(g, g)), a, b);
                        }
                        hi[j] = pack_half2(a, b);
                        if (TWO) {
                            const float2 y =
                                __half22float2(*reinterpret_cast<const __half2*>(&hi[j]));
                            lo[j] = pack_half2(a - y.x, b - y.y);
                        }
                    } else {
                        hi[j] = pack_bf16x2(a, b);
                        if (TWO)
                            lo[j] = pack_bf16x2(a - bf16lo(hi[j]), b - bf16hi(hi[j]));
                    }
                }
                tmem_st16(tS + 16 * k, hi);
                if (TWO)
                    tmem_st16(tS + 64 + 16 * k, lo);
            }
            float s0, s1, s2, s3;
            f2unpack(sum[0], s0, s1);
            f2unpack(sum[1], s2, s3);
            l += (s0 + s1) + (s2 + s3);
            tmem_st_wait();
            // V's rows that not everyone sees (TILES = 2: the first group's weights are
            // waited for before either product with this tile)
            if (masked && (TILES == 1 || w == 0)) {
                const uint32_t at = 2 * gt + 1, vs = at % C::kSlots;
                ok = mbar_wait(&sh.full[vs], (at / C::kSlots) & 1, wctx, 34);
                if (!__all_sync(0xffffffffu, ok))
                    return;
                mend_values<D, F8>(p, sh, run, slots + vs * C::kTileBytes, base, rit, missing, seg);
            }
            tc_fence_before();
            mbar_arrive(&sh.p_full[w]);
        }
        // ---- the segment's rows
        float n0 = N, d0 = F8 ? Dd : 0.f;
        const bool had[2] = {TILES == 2 || run.nt > 1 || ((gt - 1) & 1) == 0,
                             TILES == 2 || run.nt > 1 || ((gt - 1) & 1) == 1};
        if (TILES == 1) {
            sh.n[seg & 1][w][rit] = n0;
            sh.l[seg & 1][w][rit] = l;
            if (F8)
                sh.d[seg & 1][w][rit] = d0;
        }
        bool ok = mbar_wait(&sh.o_full, seg & 1, wctx, 35);
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&sh.meet);
        ok = ok && mbar_wait(&sh.meet, met, wctx, 36);
        met ^= 1;
        if (!__all_sync(0xffffffffu, ok))
            return;
        tc_fence_after();
        if (threadIdx.x < 32) {  // for the segment after the next (see `bad`)
            sh.bad[(seg + 2) % 3][lane] = 0;
            if (lane == 0)
                sh.any_bad[(seg + 2) % 3] = 0;
        }
        float fw[2] = {1.f, 1.f};
        if (TILES == 1) {
            const float na = sh.n[seg & 1][0][rit], nb = sh.n[seg & 1][1][rit];
            const float nx = fmaxf(na, nb);
            float da = na - nx, db = nb - nx, dx = 0.f;
            l = sh.l[seg & 1][0][rit] * ex2(da) + sh.l[seg & 1][1][rit] * ex2(db);
            if (F8) {
                da += sh.d[seg & 1][0][rit];
                db += sh.d[seg & 1][1][rit];
                dx = fmaxf(da, db);
            }
            fw[0] = ex2(da - dx);
            fw[1] = ex2(db - dx);
            n0 = nx;
            d0 = dx;
        }
        const bool whole = run.nt == run.tiles;
        const int64_t slot = 2 * (int64_t)blockIdx.x + (run.tile0 == 0 ? 1 : 0);
        const int64_t prow = slot * C::kRows + (TILES == 2 ? w * kTreeRows : 0) + rit;
        const int64_t orow = ((int64_t)run.b * p.Hq + run.h * p.G + gh) * p.T + tq;
        const float2 inv = row_factors<D, F8>(d0, l);
        // TILES = 1: the groups take half of the features each
        constexpr int kCols = TILES == 1 ? D / 2 : D;
#pragma unroll 1
        for (int c0 = TILES == 1 ? w * kCols : 0, end = c0 + kCols; c0 < end; c0 += 32) {
            float o[32];
            uint32_t t[32];
#pragma unroll
            for (int k = 0; k < 32; ++k)
                o[k] = 0.f;
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                if (TILES == 2 ? a != w : !had[a])
                    continue;
                tmem_ld32(tO + a * D + c0, t);
                tmem_ld_wait();
                tmem_reg_fence32(t);
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    o[k] = TILES == 1 ? fmaf(fw[a], __uint_as_float(t[k]), o[k])
                                      : __uint_as_float(t[k]);
            }
            if (!valid)
                continue;
            if (__builtin_expect(sh.any_bad[seg % 3], 0)) {
                float y[32];
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    y[k] = o[k];
                add_apart<D, F8>(p, run, sh.bad[seg % 3], mask, gh, tq, n0, d0, c0, y);
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    o[k] = y[k];
            }
            if (!whole) {
                float4* to = reinterpret_cast<float4*>(p.part_o + prow * D + c0);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    to[k] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                continue;
            }
#pragma unroll
            for (int k = 0; k < 32; ++k)
                o[k] = F8 ? o[k] * inv.x * inv.y : o[k] * inv.x;
            if (p.o_fp32) {
                float4* to = reinterpret_cast<float4*>((float*)p.o + orow * D + c0);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    to[k] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
            } else {
                uint4* to = reinterpret_cast<uint4*>((__nv_bfloat16*)p.o + orow * D + c0);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    to[k] = make_uint4(pack_bf16x2(o[8 * k], o[8 * k + 1]),
                                       pack_bf16x2(o[8 * k + 2], o[8 * k + 3]),
                                       pack_bf16x2(o[8 * k + 4], o[8 * k + 5]),
                                       pack_bf16x2(o[8 * k + 6], o[8 * k + 7]));
            }
        }
        tc_fence_before();
        mbar_arrive(&sh.o_empty);
        if (valid && (TILES == 2 || w == 0)) {
            if (whole)
                p.lse[orow] = row_lse(n0, l);
            else
                p.part_ndl[prow] = make_float4(n0, d0, l, 0.f);
        }
        if (!whole && run.tile0 == 0) {
            // the group's blocks after this one that hold the rest: up to the last tile's
            const long long last = run.w + p.segment_cost + run.tiles - 1;
            info = make_int4(run.b, run.h * p.row_groups + run.rg,
                             block_of(p, sh, last) - sh.block, run.n);
        }
    }
    if (threadIdx.x == 0)
        p.info[blockIdx.x] = info;
}

template <int D, bool F8, int TILES, bool TWO>
__global__ void __launch_bounds__(Cfg<D, F8, TILES>::kThreads, 1)
    decode_tree_kernel(const __grid_constant__ CUtensorMap tk,
                       const __grid_constant__ CUtensorMap tv, const __grid_constant__ TreeParams p)
{
    using C = Cfg<D, F8, TILES>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    Shared<D, F8, TILES>& sh = *reinterpret_cast<Shared<D, F8, TILES>*>(smem + C::kShared0);
    const uint32_t qs = smem_u32(smem) + C::kQ0, slots = smem_u32(smem) + C::kSlot0;
    const uint32_t raw = smem_u32(smem) + C::kRaw0;
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        sh.abort = 0;
        for (int s = 0; s < C::kSlots; ++s) {
            mbar_init(&sh.full[s], F8 ? 4 : 1);
            mbar_init(&sh.empty[s], 1);
        }
        for (int s = 0; s < C::kRaw; ++s) {
            mbar_init(&sh.raw_full[s], 1);
            mbar_init(&sh.raw_empty[s], 4);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sh.s_full[s], 1);
            mbar_init(&sh.p_full[s], 128);
        }
        mbar_init(&sh.o_full, 1);
        mbar_init(&sh.o_empty, 256);
        mbar_init(&sh.q_full, 2);
        mbar_init(&sh.q_empty, F8 ? 9 : 1);
        for (int s = 0; s < kRuns; ++s) {
            mbar_init(&sh.run_full[s], 1);
            mbar_init(&sh.run_empty[s], C::kReaders);
        }
        for (int s = 0; s < kRing; ++s)
            mbar_init(&sh.info_full[s], 1);
        mbar_init(&sh.meet, 8);
        fence_barrier_init();
        prefetch_tmap(&tk);
        prefetch_tmap(&tv);
        p.info[blockIdx.x] = make_int4(0, 0, 0, 0);  // for a block that gives up
    }
    if (threadIdx.x < 96)
        sh.bad[threadIdx.x / 32][threadIdx.x % 32] = 0;
    if (threadIdx.x < 3)
        sh.any_bad[threadIdx.x] = 0;
    if (warp == 8) {
        tmem_alloc(&sh.tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    find_range<C::kThreads>(p, sh);  // also orders the initialisation
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    const WaitCtx wctx{&sh.abort, p.c.status, p.timeout_ns};
    if (warp < 8) {
        reg_alloc<C::kRegsMath>();
        softmax<D, F8, TILES, TWO>(p, sh, slots, tmem, wctx);
    } else if (warp < 12) {
        reg_dealloc<C::kRegsCtl>();
        if (warp == 8) {
            multiply<D, F8, TILES, TWO>(sh, qs, slots, tmem, wctx);
        } else if (warp == 9) {
            produce<D, F8, TILES>(p, sh, F8 ? raw : slots, tk, tv, wctx);
            if (*wctx.abort_flag) {
                // let copies in flight land before the block's shared memory goes
                const uint64_t t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < 2000000ull) {
                }
            }
        } else {
            load_queries<D, F8, TILES>(p, sh, qs, wctx);
        }
    } else if constexpr (F8) {
        reg_dealloc<C::kRegsConv>();
        convert<D, TILES>(p, sh, slots, raw, wctx);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Rows of the segments that several blocks share: block c holds such a segment's
// beginning, the info[c].z blocks of its group after it the rest.  One warp a row.
template <int D, bool F8, int ROWS>
__global__ void __launch_bounds__(256) merge_kernel(const __grid_constant__ TreeParams p)
{
    const int4 info = p.info[blockIdx.x];
    const int k = info.z + 1;
    if (info.z <= 0)
        return;
    const int32_t h = info.y / p.row_groups, r0 = (info.y - h * p.row_groups) * ROWS;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int own = 2 * blockIdx.x, step = 2 * p.row_groups;
    auto slot = [&](int i) -> int64_t { return i == 0 ? own + 1 : own + i * step; };
    constexpr int V = D / 32;  // features of a lane
    for (int r = blockIdx.y * 8 + warp; r < ROWS && r0 + r < p.G * p.T; r += gridDim.y * 8) {
        int32_t gh, tq;
        split_row(p, r0 + r, gh, tq);
        if (tq >= info.w)
            continue;
        float nx = kNone, dx = F8 ? -INFINITY : 0.f;
        for (int i = lane; i < k; i += 32)
            nx = fmaxf(nx, p.part_ndl[slot(i) * ROWS + r].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            nx = fmaxf(nx, __shfl_xor_sync(0xffffffffu, nx, o));
        if (F8) {
            for (int i = lane; i < k; i += 32) {
                const float4 y = p.part_ndl[slot(i) * ROWS + r];
                dx = fmaxf(dx, (y.x - nx) + y.y);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                dx = fmaxf(dx, __shfl_xor_sync(0xffffffffu, dx, o));
        }
        float L = 0.f, acc[V] = {};
        for (int c = 0; c < k; c += 32) {
            float4 y = make_float4(kNone, 0.f, 0.f, 0.f);
            if (c + lane < k)
                y = p.part_ndl[slot(c + lane) * ROWS + r];
            const float wt = ex2((y.x - nx) + (y.y - dx));
            L += y.z * ex2(y.x - nx);
            const int end = min(32, k - c);
#pragma unroll 4
            for (int i = 0; i < end; ++i) {
                const float wi = __shfl_sync(0xffffffffu, wt, i);
                const float* from = p.part_o + (slot(c + i) * ROWS + r) * D + lane * V;
#pragma unroll
                for (int v = 0; v < V; ++v)
                    acc[v] = fmaf(wi, from[v], acc[v]);
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            L += __shfl_xor_sync(0xffffffffu, L, o);
        const float2 inv = row_factors<D, F8>(dx, L);
        const int64_t at = ((int64_t)info.x * p.Hq + h * p.G + gh) * p.T + tq;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            acc[v] = F8 ? acc[v] * inv.x * inv.y : acc[v] * inv.x;
            if (p.o_fp32)
                ((float*)p.o)[at * D + lane * V + v] = acc[v];
        }
        if (!p.o_fp32)
#pragma unroll
            for (int v = 0; v < V; v += 2)
                reinterpret_cast<uint32_t*>((__nv_bfloat16*)p.o + at * D + lane * V)[v / 2] =
                    pack_bf16x2(acc[v], acc[v + 1]);
        if (lane == 0)
            p.lse[at] = row_lse(nx, L);
    }
}

template <int D, bool F8, int TILES, bool TWO>
cudaError_t launch(const CUtensorMap& tk, const CUtensorMap& tv, TreeParams& p, int num_sms,
                   cudaStream_t stream)
{
    using C = Cfg<D, F8, TILES>;
    static_assert(kSmem<D, F8, TILES> <= 232448, "shared memory");
    cudaError_t e = cudaFuncSetAttribute(decode_tree_kernel<D, F8, TILES, TWO>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kSmem<D, F8, TILES>);
    if (e != cudaSuccess)
        return e;
    // a block an SM, no more than there can be pieces
    const int64_t segments = (int64_t)p.c.B * p.c.Hkv;  // of one row group
    const int32_t longest = max(1, ceil_div(p.c.max_pages * p.c.page, kTile));
    p.whole = longest <= kWhole;
    const int64_t pieces = min(segments, (int64_t)kTreeMaxCtas) * (p.whole ? 1 : longest);
    p.row_groups = ceil_div(p.G * p.T, C::kRows);
    const int most = min(kTreeMaxCtas, num_sms);
    p.line_blocks = (int)min((int64_t)max(1, most / p.row_groups), pieces);
    const int grid = p.line_blocks * p.row_groups;
    p.segment_cost = 2;
    decode_tree_kernel<D, F8, TILES, TWO>
        <<<grid, C::kThreads, kSmem<D, F8, TILES>, stream>>>(tk, tv, p);
    e = cudaGetLastError();
    if (e != cudaSuccess || p.whole)
        return e;
    const int rows = min(C::kRows, p.G * p.T);
    merge_kernel<D, F8, C::kRows><<<dim3(grid, (rows + 7) / 8), 256, 0, stream>>>(p);
    return cudaGetLastError();
}

template <int D, bool F8>
cudaError_t launch_rows(const CUtensorMap& tk, const CUtensorMap& tv, TreeParams& p, int num_sms,
                        cudaStream_t stream)
{
    const bool one = p.G * p.T <= kTreeRows;
    if (F8 && !p.o_fp32)  // (see "Rounding" above)
        return one ? launch<D, F8, 1, !F8>(tk, tv, p, num_sms, stream)
                   : launch<D, F8, 2, !F8>(tk, tv, p, num_sms, stream);
    return one ? launch<D, F8, 1, true>(tk, tv, p, num_sms, stream)
               : launch<D, F8, 2, true>(tk, tv, p, num_sms, stream);
}

}  // namespace tree

cudaError_t launch_decode_tree(const CUtensorMap& tk, const CUtensorMap& tv, TreeParams& p,
                               int num_sms, cudaStream_t stream)
{
    if (p.c.e4m3)
        return p.c.d == 128 ? tree::launch_rows<128, true>(tk, tv, p, num_sms, stream)
                            : tree::launch_rows<64, true>(tk, tv, p, num_sms, stream);
    return p.c.d == 128 ? tree::launch_rows<128, false>(tk, tv, p, num_sms, stream)
                        : tree::launch_rows<64, false>(tk, tv, p, num_sms, stream);
}

}  // namespace dfa
