// dfa_tree_attn.cu -- attention of trees of drafted tokens over a paged key/value cache, on
// the tensor cores: the nodes of a tree, times the query heads that share a key/value
// head, against the rows of their sequence.
//
// Method.  With keys k_j = s_j c_j and values v_j = u_j w_j (codes and scales; 1 for bf16
// cells), a query row has x_j = scale log2(e) s_j (q . c_j) and
//   O = 2^D (sum_j 2^(x_j - N + log2 u_j - D) w_j) / (sum_j 2^(x_j - N)),
//   LSE = ln 2 (N + log2 sum),
// with N the running maximum of the scores, and D that of the weights' exponents beyond it
// (0 for bf16 cells), so that weights fit their type whatever the scales are.  Scores far
// from zero are rounded to fp32 before N is taken off them, as N was when it was one of
// them: the difference is exact however large both are.  Weights are the sum's terms times
// 2^(log2 u_j - D), where every u_j of a tile is in [2^-40, 2^40] and D is not far below
// that, and else powers of their own.
//
// What a node sees: every row before the tree, and of the tree's rows those whose bits
// its mask has.  Only tiles that reach into the tree or over the sequence's end look at
// masks; a row of the tile is 128 bits.
//
// A block (one an SM) keeps 128 query rows and walks over 128-key tiles of the cache:
//   warp 9       pages by TMA into a ring of K and V tiles, 128-byte swizzle;
//   warps 12-15  (8-bit cells) those to fp16, in the same layout;
//   warp 11      the next segment's queries (8-bit cells: fp16 relative to a power of two
//                of the row: exact but for elements below 2^-31 of its largest one);
//   warps 8, 10  S = Q K^T into TMEM, O += P V with P from TMEM (over S's columns);
//   warps 0-3    softmax of the tile's first 64 keys, warps 4-7 of the others, a thread a
//                row, each with an N, D, sum and O of its own, joined at the segment's end.
//                O is rescaled in TMEM when D (or N) has to rise.
// S has two buffers (three for d = 64): the next tile's scores are there when a tile's
// softmax ends.
//
// Bound: bf16 cells by HBM (64 ragged sequences up to 8K 182 us, 6.0 TB/s; 4 sequences up to
// 32K, 128 rows a head 70 us, 73 % of DRAM's peak with start and tail); those of d = 64 with
// more than 64 rows a head, which have half the bytes for the same softmax, by each group's
// way from scores to weights (128K rows 72 us, where HBM takes 40: half of the issue slots, half
// of DRAM's peak and a third of the tensor pipe's cycles are used).  8-bit cells of d = 128
// by shared memory, whose 224 KB a tile (arriving, converted, read by the products) take 1800
// of 2000 to 2150 clk: 42 % of its pipe's cycles are loads and stores and 30 % the products',
// start and tail among them (8 sequences up to 16K, 240 rows a head: 96 us; HBM takes 23, the
// products 38).
//
// Work: (sequence, head, row group) segments form one line, cut by cost over a grid of
// one block an SM: a block's range covers whole segments, whose result it writes, and up
// to two cut ones, whose partials merge_kernel joins.  The lengths are read on the
// device, so a captured graph follows them.
//
// Rounding: weights as two bf16 terms (2^-17) for bf16 cells, with an fp32 output and at
// most 64 query rows a head as three (2^-25; with more there is no room in TMEM beside
// them); for 8-bit cells as one fp16 term (2^-11) with a bf16 output, as two (2^-22) with an
// fp32 one.  Sums, maxima and O in fp32; see kChain.
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
constexpr int kRuns = 2;                  // segments that are announced ahead
// N rises when a term exceeds 2^grow.  For bf16 weights, which are the terms and which values
// up to 2^120 over the number of rows are multiplied by, that costs a pass over O (128K rows
// 71.7 us; with 60, which values above 2^68 do not bear, 70.6).  8-bit cells have D for their
// weights, and terms of 2^60 come nowhere near fp32's end.
constexpr float grow(bool f8) { return f8 ? 60.f : 8.f; }
// fp16 weights: D is set `head` below the largest exponent, and set anew, with a pass over
// O, when a weight exceeds 2^kTop.  Between the two is room for larger weights to come;
// `head` is what small ones behind a large one have left: half a step of fp16's subnormals
// is 2^-33 of the largest weight, 2^-16 for 128K of them together, with 8 (fp32
// outputs), 2^-29 and 2^-12 at worst with 4 (bf16 outputs, which are rounded to 2^-9; trees
// of 60 over 16K 100 us in place of 103, 15 of 40 tiles having made a pass over O before):
// head() below.
constexpr float kTop = 15.f;
// A product adds to O by cutting off what fp32 does not hold, which makes O smaller each
// time, in the end by 2^-24 of it for every other product.  So a sum of so many tiles is set
// apart (in the workspace; the next begins at 0) and added at the segment's end.  fp32
// outputs: off by 2.7e-6 in place of 3.5e-6 after 128K rows, 54 tiles a block, for 71 us in
// place of 67; every 16 tiles 2.5e-6 and 73 us.  bf16 outputs: a batch of contexts of 1M rows,
// 8192 tiles a block, was smaller by up to 2.4e-3, more than rounding takes; 256 tiles leave
// less than 3e-4, of which fp16 weights have their part.  (Weights in one term: a kernel with
// chains is 1 to 2 % slower, 4 sequences of 128 rows 73.6 us against 72.0, and is taken where
// a sequence can have more tiles than that.)
constexpr int kChain = 32, kLongChain = 256;
constexpr float kNone = -FLT_MAX;         // running maximum before the first key
constexpr float kFar = 1048576.f;         // scores as far from zero are rounded before N is
                                          // taken off them (else both in one operation: N,
                                          // rounded, is then off by 2^-4 at most)
// Terms times 2^(log2 u_j - D) are weights while |log2 u_j| is at most kNear and D at least
// kLow (which tiny values before this tile leave behind): the factor is then at most 2^100, so
// that it is finite, and a term that vanishes (below 2^-126) has no weight that fp16 holds.
constexpr float kNear = 40.f, kLow = -60.f;
constexpr float kLn2 = 0.69314718055994531f;
// Where no sequence can be longer than so many tiles, segments are not cut and there is
// nothing to merge.
constexpr int kWhole = 2;
constexpr int kSiteShared = 109;         // of DFA_ERR_BOUNDS in DevStatus::where
constexpr uint32_t kWideTile = 256;       // flag of a tile, beside the missing pages' bits

// A run of tiles [tile0, tile0 + nt) of one segment: key/value head h, row group rg of
// sequence b, which has len rows, n nodes and that many tiles.
struct Piece {
    int32_t b, h, rg, len, n;
    int32_t tile0, nt, tiles;
    long long w;  // the segment's first unit on the line
};

// How weights are held: in one term; in two, side by side in the operand's columns; in two
// in its rows, where at most 64 of the 128 rows have queries: rows r and r + 64 are the
// same query's, and the second row's weights are what the first's leave; in three: two in
// the rows, the third in the first's columns.  kSplit: one term, but rows r and r + 64 are
// the same query's, each with half of the keys (and zeros, N, D and O of its own).
enum Terms { kOne, kColumns, kLanes, kThree, kSplit };
constexpr bool by_rows(Terms t) { return t == kLanes || t == kThree || t == kSplit; }
constexpr float head(Terms t) { return t == kOne || t == kSplit ? 4.f : 8.f; }
constexpr int chunks(Terms t) { return t == kSplit ? 2 : 4; }  // of 16 keys, a row's of a tile
constexpr bool by_columns(Terms t) { return t == kColumns || t == kThree; }

template <int D, bool F8>
struct Cfg {
    static constexpr int kThreads = F8 ? 512 : 384;
    static constexpr int kTileBytes = kTile * D * 2;      // a K, V or Q tile of 16-bit elements
    static constexpr int kRawBytes = kTile * D;
    // buffers of S: as many as TMEM has room for beside two O
    static constexpr int kS = D == 128 ? 2 : 3;
    static constexpr int kO0 = kS * 128;                  // column of O
    // slots of K and V tiles: K's are free when its scores are there, V's two tiles later
    static constexpr int kK = F8 ? (D == 128 ? 1 : 2) : (D == 128 ? 2 : 4);
    static constexpr int kV = F8 ? (D == 128 ? 2 : 3) : (D == 128 ? 3 : 5);
    static constexpr int kRaw = !F8 ? 0 : D == 128 ? 3 : 6;
    static constexpr int kK0 = 2 * kTileBytes;            // behind two segments' queries
    static constexpr int kV0 = kK0 + kK * kTileBytes;
    static constexpr int kRaw0 = kV0 + kV * kTileBytes;
    static constexpr int kShared0 = kRaw0 + kRaw * kRawBytes;
    // What a segment costs a block beside its tiles, in tiles.  Measured: bf16 (1, 2, 3, 4),
    // 64 ragged sequences of 16 nodes 194.4, 187.0, 188.7, 191.9 us; 8 bits (3, 5, 8), 8
    // sequences of 240 rows 103.7, 102.5, 103.2, 4 of 128 rows 74.7, 73.5, 73.8, but 4 of
    // 16 rows 66.0, 66.8, 67.7.
    static constexpr int segment_cost(int rows) { return !F8 ? 2 : rows > 64 ? 5 : 3; }
    static constexpr int kReaders = 8 + 1 + 2 + (F8 ? 4 : 0);  // warps that read a run
};

template <bool F8>
struct TileInfo {
    float2 scale[F8 ? 8 : 1];  // per page: K's scale, log2 of V's
    uint32_t flags;            // pages that are not there; kWideTile
};

template <int D, bool F8>
struct Shared {
    using C = Cfg<D, F8>;
    uint64_t k_full[C::kK], k_empty[C::kK], v_full[C::kV], v_empty[C::kV];
    uint64_t raw_full[F8 ? C::kRaw : 1], raw_empty[F8 ? C::kRaw : 1];
    uint64_t s_full[C::kS], s_free[C::kS], p_full[2][C::kS], o_empty, q_full[2], q_empty[2], q_first;
    uint64_t run_full[kRuns], run_empty[kRuns], info_full[kRing], meet, handed;
    Piece run[kRuns];
    TileInfo<F8> info[kRing];
    long long w0, w1, base, each, rest;
    int32_t b, block, rows, nodes;
    uint32_t tmem, abort;
    union {
        long long warp_sum[16];  // while the range is found
        uint32_t bad[3][32];     // nodes whose values are not finite
    };
    uint32_t any_bad[3];
    float qf[F8 ? 2 : 1][F8 ? kTreeRows : 1];             // score factors of the rows
    // of the two groups: N (before, what is set apart of O is to be multiplied by), sum, D
    float n[2][kTreeRows], l[2][kTreeRows], d[F8 ? 2 : 1][F8 ? kTreeRows : 1];
};

template <int D, bool F8>
constexpr int kSmem = Cfg<D, F8>::kShared0 + (int)sizeof(Shared<D, F8>);

// mbar_wait with its loop out of the way: the roles' inner loops are to fit the first
// instruction caches, which they share.
__device__ __noinline__ bool wait_on(uint64_t* bar, uint32_t parity, const WaitCtx& w, int where)
{
    return mbar_wait(bar, parity, w, where);
}

__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, const WaitCtx& w, int where)
{
    return mbar_try_wait(bar, parity) || wait_on(bar, parity, w, where);
}

// columns of a row's 8 words
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
        : "memory");
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

// Out of line, as what follows that is not in an inner loop: the code that a block goes
// through once or once a segment comes from far away, 128 bytes at a time.
__device__ __forceinline__ int2 rows_of(const TreeParams& p, int32_t b)
{
    int32_t len, n;
    seq_rows(p.c, p.q_lens, p.T, b, len, n);
    return make_int2(len, n);
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
        len = sh.rows, n = sh.nodes;
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
                    const int2 r = rows_of(p, b);
                    len = r.x, n = r.y;
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
        sh.rows = 0;
        sh.nodes = 0;
        sh.block = block;
        sh.base = 0;
    }
    const int32_t b0 = threadIdx.x * chunk, b1 = min(b0 + chunk, p.c.B);
    long long sum = 0;
    int2 r = make_int2(0, 0);  // of the thread's last sequence
    for (int32_t b = b0; b < b1; ++b) {
        r = rows_of(p, b);
        const int32_t tiles = tiles_of(r.x, r.y);
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
            if (chunk > 1)
                r = rows_of(p, b);
            const int32_t tiles = tiles_of(r.x, r.y);
            const long long t = tiles ? (long long)(tiles + p.segment_cost) * per_seq : 0;
            if (w0 < base + t) {
                sh.b = b;
                sh.base = base;
                sh.rows = r.x;
                sh.nodes = r.y;
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
    const bool ok = wait(&sh.run_full[seg % kRuns], (seg / kRuns) & 1, wctx, where);
    if (!__all_sync(0xffffffffu, ok))
        return false;
    run = sh.run[seg % kRuns];
    __syncwarp();
    if ((threadIdx.x & 31) == 0)
        mbar_arrive(&sh.run_empty[seg % kRuns]);
    return run.nt > 0;
}

// Is the output fp32?  (What launch_terms leaves open is known to the compiler.)
template <bool F8, Terms TERMS>
__device__ __forceinline__ bool is_fp32(const TreeParams& p)
{
    if (TERMS == kOne || TERMS == kSplit || (TERMS == kLanes && !F8))
        return false;
    return F8 || TERMS == kThree || p.o_fp32;
}

// The tile i of a segment begins a chain where i & this is 0.
template <bool F8, Terms TERMS, bool LONG>
__device__ __forceinline__ int32_t chain_mask(const TreeParams& p)
{
    return !LONG ? INT32_MAX : (is_fp32<F8, TERMS>(p) ? kChain : kLongChain) - 1;
}

// A place in a ring of SLOTS, and the phase that its barriers are in.
template <int SLOTS>
struct Ring {
    uint32_t at = 0, phase = 0;
    __device__ __forceinline__ void next()
    {
        if (++at == SLOTS) {
            at = 0;
            phase ^= 1;
        }
    }
};

// ---------------------------------------------------------------------------
// producer: the tiles' pages, and what there is to know of them
// ---------------------------------------------------------------------------
template <int D, bool F8>
__device__ __forceinline__ void produce(const TreeParams& p, Shared<D, F8>& sh,
                                        uint32_t smem, const CUtensorMap& tk,
                                        const CUtensorMap& tv, const WaitCtx& wctx)
{
    using C = Cfg<D, F8>;
    constexpr int kPlanes = F8 ? 1 : D / 64;            // boxes side by side
    constexpr int kBoxRow = F8 ? D : 128;               // bytes of a box's row
    constexpr int kBytes = F8 ? C::kRawBytes : C::kTileBytes;
    const int lane = threadIdx.x & 31;
    const int32_t page = p.c.page;
    const int32_t per_tile = kTile / page;
    Ring<F8 ? C::kRaw : C::kK> kr;  // 8-bit cells: of K and V in turn
    Ring<C::kV> vr;
    uint32_t seg = 0, gt = 0;
    Walk wk;
    wk.start(p, sh, blockIdx.x - sh.block * p.row_groups);
    bool more = wk.next(p);
    // Table entry of this lane's page of the 32 from page `win` on; -1: none.
    auto entry = [&](const Walk& x, int32_t win) {
        const int32_t end = ceil_div(min(x.len, (x.tile0 + x.nt) * kTile), page);
        return win + lane < end ? page_entry(p.c, x.b, win + lane) : -1;
    };
    // Segment `seg` to all readers, or that there is none.
    auto announce = [&](uint32_t seg, const Piece& run, bool end) {
        const bool ok = wait(&sh.run_empty[seg % kRuns], (seg / kRuns + 1) & 1, wctx, 51);
        if (!__all_sync(0xffffffffu, ok))
            return false;
        if (lane == 0) {
            sh.run[seg % kRuns] = run;
            if (end)
                sh.run[seg % kRuns].nt = 0;
            mbar_arrive(&sh.run_full[seg % kRuns]);
        }
        return true;
    };
    int32_t next_id = more ? entry(wk, (wk.tile0 * kTile) >> p.c.page_log2) : -1;
    if (!announce(0, wk, !more))
        return;
    for (; more; ++seg) {
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
                uint64_t* full = F8 ? &sh.raw_full[kr.at] : kv ? &sh.v_full[vr.at] : &sh.k_full[kr.at];
                uint64_t* empty =
                    F8 ? &sh.raw_empty[kr.at] : kv ? &sh.v_empty[vr.at] : &sh.k_empty[kr.at];
                const uint32_t slot = smem + (F8 ? C::kRaw0 + kr.at * kBytes
                                              : kv ? C::kV0 + vr.at * kBytes
                                                   : C::kK0 + kr.at * kBytes);
                // (passes at once in the first round: the phase before the barrier's first)
                const bool ok = wait(empty, (F8 || !kv ? kr.phase : vr.phase) ^ 1, wctx, 50);
                if (!__all_sync(0xffffffffu, ok))
                    return;
                if (lane == 0)
                    mbar_expect(full, __popc(boxes) * (page * D * (F8 ? 1 : 2)));
                __syncwarp();
                if (load) {
                    const uint32_t dst = slot + lane * page * kBoxRow;
#pragma unroll
                    for (int pl = 0; pl < kPlanes; ++pl)
                        tma_load_4d(dst + pl * kTile * 128, kv ? &tv : &tk, full, pl * 64, 0, h, my);
                }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(full);
                if (F8 || !kv)
                    kr.next();
                else
                    vr.next();
            }
            // What the softmax has to know.  (A tile's entry is written anew kRing tiles
            // later, when the ring's slots say that its softmax is long done.)
            TileInfo<F8>& info = sh.info[gt % kRing];
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
            if (F8 && lane < per_tile)
                info.scale[lane] = make_float2(load ? my_ks : 1.f, lu);
            const uint32_t missing = ~boxes & ((1u << per_tile) - 1);
            if (lane == 0)
                info.flags = missing | (wide ? kWideTile : 0u);
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sh.info_full[gt % kRing]);
            if (i == look) {
                more_next = nx.next(p);
                next_id = more_next ? entry(nx, (nx.tile0 * kTile) >> p.c.page_log2) : -1;
                // (at once: its queries take one warp several tiles' time.  All readers have
                // the segment before this one, or what they need to come to it.)
                if (!announce(seg + 1, nx, !more_next))
                    return;
            }
        }
        wk = nx;
        more = more_next;
    }
}

// ---------------------------------------------------------------------------
// queries of the segments
// ---------------------------------------------------------------------------
// Queries of a segment into its buffer, by WARPS warps: all on their way at once, then,
// for 8-bit cells, each lane turns what it copied.  (Rows without a query stay as they
// are: nobody looks at what comes of them.)
template <int D, bool F8, Terms TERMS, int WARPS>
__device__ __forceinline__ void copy_queries(const TreeParams& p, Shared<D, F8>& sh, uint32_t qs,
                                             const Piece& run, uint32_t seg, int warp)
{
    using C = Cfg<D, F8>;
    constexpr int kPerRow = D / 8;                 // lanes of a row, 8 elements each
    constexpr int kRowsAt = 32 / kPerRow * WARPS;  // rows at a time
    const int lane = threadIdx.x & 31, c = lane % kPerRow;
    const int32_t first = warp * (32 / kPerRow) + lane / kPerRow;
    const uint32_t to = qs + (seg & 1) * C::kTileBytes + (c >> 3) * (kTreeRows * 128);
    const int32_t rows = min(kTreeRows, p.G * p.T - run.rg * kTreeRows);
    const __nv_bfloat16* q =
        (const __nv_bfloat16*)p.q.p + run.b * p.q.sb + (int64_t)run.h * p.G * p.q.sh + c * 8;
#pragma unroll 4
    for (int32_t row = first; row < rows; row += kRowsAt) {
        int32_t gh, tq;
        split_row(p, run.rg * kTreeRows + row, gh, tq);
        if (tq < run.n)
#pragma unroll
            for (int i = 0; i < (by_rows(TERMS) && !F8 ? 2 : 1); ++i)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                 to + sw128_offset(row + 64 * i, c & 7)),
                             "l"(q + gh * p.q.sh + tq * p.q.sl)
                             : "memory");
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (F8) {
        constexpr int kBatch = 8 / (WARPS == 1 ? 1 : D == 128 ? 1 : 2);  // rows a lane at a time
        for (int32_t r0 = first; r0 - first < rows; r0 += kBatch * kRowsAt) {
            uint4 x[kBatch];
            float amax[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                x[k] = lds128(to + sw128_offset(r0 + k * kRowsAt, c & 7));
                amax[k] = fmaxf(fmaxf(fmaxf(fabsf(bf16lo(x[k].x)), fabsf(bf16hi(x[k].x))),
                                      fmaxf(fabsf(bf16lo(x[k].y)), fabsf(bf16hi(x[k].y)))),
                                fmaxf(fmaxf(fabsf(bf16lo(x[k].z)), fabsf(bf16hi(x[k].z))),
                                      fmaxf(fabsf(bf16lo(x[k].w)), fabsf(bf16hi(x[k].w)))));
            }
#pragma unroll
            for (int o = 1; o < kPerRow; o <<= 1)
#pragma unroll
                for (int k = 0; k < kBatch; ++k)
                    amax[k] = fmaxf(amax[k], __shfl_xor_sync(0xffffffffu, amax[k], o));
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int32_t row = r0 + k * kRowsAt;
                // the largest element to [2^14, 2^15): those down to 2^-31 of it stay exact
                const int e = min(max((int)(__float_as_uint(amax[k]) >> 23) - 127, -100), 126) - 14;
                const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
                uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w[i] = pack_half2(bf16lo(w[i]) * inv, bf16hi(w[i]) * inv);
                if (row < rows)
#pragma unroll
                    for (int i = 0; i < (by_rows(TERMS) ? 2 : 1); ++i) {
                        st_shared_v4(to + sw128_offset(row + 64 * i, c & 7), w[0], w[1], w[2], w[3]);
                        if (c == 0)
                            sh.qf[seg & 1][row + 64 * i] =
                                p.scale_log2 * __uint_as_float((uint32_t)(127 + e) << 23);
                    }
            }
        }
    }
    fence_proxy_async_smem();
    __syncwarp();
}

// (The first segment's are copied by the softmax warps, who would wait for them.)
template <int D, bool F8, Terms TERMS>
__device__ __forceinline__ void load_queries(const TreeParams& p, Shared<D, F8>& sh, uint32_t qs,
                                             const WaitCtx& wctx)
{
    Piece run;
    for (uint32_t seg = 0; next_run(sh, seg, run, wctx, 53); ++seg) {
        const bool ok = wait(&sh.q_empty[seg & 1], ((seg >> 1) & 1) ^ 1, wctx, 54);
        if (!__all_sync(0xffffffffu, ok))
            return;
        if (seg > 0)
            copy_queries<D, F8, TERMS, 1>(p, sh, qs, run, seg, 0);
        if ((threadIdx.x & 31) == 0)
            mbar_arrive(&sh.q_full[seg & 1]);
    }
}

// ---------------------------------------------------------------------------
// 8-bit cells to fp16
// ---------------------------------------------------------------------------
// A warp takes 32 rows.  Eight lanes at a time read 16 bytes each and write twice that,
// which the swizzles keep free of bank conflicts where the two rows they are of differ in
// bits 0 and 2 (128-byte rows), or in bit 0 (64-byte rows, two to a line).
template <int D>
__device__ __forceinline__ void convert(Shared<D, true>& sh, uint32_t smem, const WaitCtx& wctx)
{
    using C = Cfg<D, true>;
    const int warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
    const int sub = lane & 7, g = lane >> 3;
    // offsets of the thread's first 16 codes (128-byte rows: of either half of a row), and
    // of the 16-byte chunks that they become; then every 8 rows
    uint32_t src[D / 64], dst[D / 64][2];
#pragma unroll
    for (int half = 0; half < D / 64; ++half) {
        const uint32_t row = warp * 32 + (D == 128 ? ((sub >> 2) ? g ^ 5 : g) : g * 2 + (sub >> 2));
        const uint32_t ch = (sub & 3) + 4 * half;
        src[half] = D == 128 ? row * 128 + ((ch ^ (row & 7)) << 4)
                             : row * 64 + ((ch ^ ((row >> 1) & 3)) << 4);
#pragma unroll
        for (int e = 0; e < 2; ++e)
            dst[half][e] = half * (kTile * 128) + sw128_offset(row, 2 * (sub & 3) + e);
    }
    Ring<C::kRaw> rr;
    Ring<C::kK> kr;
    Ring<C::kV> vr;
    Piece run;
    for (uint32_t seg = 0; next_run(sh, seg, run, wctx, 55); ++seg) {
        for (int32_t i = 0; i < 2 * run.nt; ++i) {
            const bool is_v = i & 1;
            bool ok = wait(&sh.raw_full[rr.at], rr.phase, wctx, 56);
            ok = ok && (is_v ? wait(&sh.v_empty[vr.at], vr.phase ^ 1, wctx, 57)
                             : wait(&sh.k_empty[kr.at], kr.phase ^ 1, wctx, 58));
            if (!__all_sync(0xffffffffu, ok))
                return;
            const uint32_t from = smem + C::kRaw0 + rr.at * C::kRawBytes;
            const uint32_t to = smem + (is_v ? C::kV0 + vr.at * C::kTileBytes
                                             : C::kK0 + kr.at * C::kTileBytes);
#pragma unroll
            for (int half = 0; half < D / 64; ++half) {
                uint4 x[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    x[k] = lds128(from + src[half] + k * 8 * D);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        st_shared_v4(to + dst[half][e] + k * 1024, e4m3x2_half2(w[2 * e] & 0xffffu),
                                     e4m3x2_half2(w[2 * e] >> 16),
                                     e4m3x2_half2(w[2 * e + 1] & 0xffffu),
                                     e4m3x2_half2(w[2 * e + 1] >> 16));
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(is_v ? &sh.v_full[vr.at] : &sh.k_full[kr.at]);
                mbar_arrive(&sh.raw_empty[rr.at]);
            }
            rr.next();
            if (is_v)
                vr.next();
            else
                kr.next();
        }
    }
}

// ---------------------------------------------------------------------------
// products, issued by a thread of one warp each, so that neither waits for the other's
// barriers
// ---------------------------------------------------------------------------
// The warps go through their loops whole, and one lane is elected at each instruction:
// descriptors and addresses are then the warp's, and stay in its uniform registers.
// Measured (clk to issue a product with both operands in shared memory, and with one in
// TMEM): 43 and 39, by one lane's loop 73 and 111.
__device__ __forceinline__ void mma_ss_one(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                           uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate));
}

__device__ __forceinline__ void mma_ts_one(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                           uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate));
}

__device__ __forceinline__ void commit_one(uint64_t* bar)
{
    asm volatile(
        "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
            smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, const WaitCtx& w,
                                         int where)
{
    return __all_sync(0xffffffffu, wait(bar, parity, w, where));
}

// S = Q K^T, as many tiles ahead of the products as there are buffers
template <int D, bool F8>
__device__ __forceinline__ void multiply_scores(Shared<D, F8>& sh, uint32_t smem,
                                                const WaitCtx& wctx)
{
    using C = Cfg<D, F8>;
    const uint64_t dQ = sdesc_sw128(smem, 16, 1024);
    const uint64_t dK = sdesc_sw128(smem + C::kK0, 16, 1024);
    Ring<C::kK> kr;
    Ring<C::kS> sr;
    Piece run;
    for (uint32_t seg = 0; next_run(sh, seg, run, wctx, 20); ++seg) {
        const uint64_t q = sdesc_add(dQ, (seg & 1) * C::kTileBytes);
        if (!wait_all(&sh.q_full[seg & 1], (seg >> 1) & 1, wctx, 21) ||
            (seg == 0 && !wait_all(&sh.q_first, 0, wctx, 21)))
            return;
        const int32_t nt = __shfl_sync(0xffffffffu, run.nt, 0);
        for (int32_t i = 0; i < nt; ++i, sr.next(), kr.next()) {
            if (!wait_all(&sh.s_free[sr.at], sr.phase ^ 1, wctx, 27) ||
                !wait_all(&sh.k_full[kr.at], kr.phase, wctx, 22))
                return;
            tc_fence_after();
            const uint64_t k = sdesc_add(dK, kr.at * C::kTileBytes);
            const uint32_t to = sr.at * 128;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
                mma_ss_one(to, sdesc_add(q, off), sdesc_add(k, off), idesc<F8>(128, false), kk > 0);
            }
            commit_one(&sh.s_full[sr.at]);
            commit_one(&sh.k_empty[kr.at]);
            if (i + 1 == nt)
                commit_one(&sh.q_empty[seg & 1]);
        }
    }
}

// O_w += P_w V, of 64 keys each
template <int D, bool F8, Terms TERMS>
__device__ __forceinline__ void multiply_values(Shared<D, F8>& sh, uint32_t smem, int32_t chain,
                                                const WaitCtx& wctx)
{
    using C = Cfg<D, F8>;
    const uint64_t dV = sdesc_sw128(smem + C::kV0, 16384, 1024);
    Ring<C::kV> vr;
    Ring<C::kS> sr;
    Piece run;
    for (uint32_t seg = 0; next_run(sh, seg, run, wctx, 28); ++seg) {
        if (!wait_all(&sh.o_empty, (seg & 1) ^ 1, wctx, 23))
            return;
        const int32_t nt = __shfl_sync(0xffffffffu, run.nt, 0);
        for (int32_t i = 0; i < nt; ++i, sr.next(), vr.next()) {
            if (!wait_all(&sh.v_full[vr.at], vr.phase, wctx, 24))
                return;
            const uint64_t v = sdesc_add(dV, vr.at * C::kTileBytes);
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                if (!wait_all(&sh.p_full[w][sr.at], sr.phase, wctx, 25 + w))
                    return;
                tc_fence_after();
                const uint32_t from = sr.at * 128 + w * 64;
#pragma unroll
                for (int kk = 0; kk < (by_columns(TERMS) ? 8 : 4); ++kk)
                    mma_ts_one(C::kO0 + w * D,
                               from + (by_columns(TERMS) ? (kk & 3) * 16 + (kk >> 2) * 8 : kk * 8),
                               sdesc_add(v, (w * 4 + (kk & 3)) * 2048), idesc<F8>(D, true),
                               ((i & chain) || kk > 0) ? 1u : 0u);
            }
            commit_one(&sh.s_free[sr.at]);
            commit_one(&sh.v_empty[vr.at]);
        }
    }
}

// ---------------------------------------------------------------------------
// softmax
// ---------------------------------------------------------------------------
// Which of the 64 keys from key `base` on a node sees: of the rows before the tree all,
// of the tree's those of its mask (NULL: none), of missing pages (from `base` on) none.
__device__ __noinline__ uint2 visible(int32_t tree0, int32_t n, int32_t words, int32_t base,
                                      const uint32_t* mask, uint32_t missing)
{
    uint32_t vis[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int32_t k0 = base + 32 * i, off = k0 - tree0;  // node of the word's first key
        uint32_t bits = off <= -32 ? ~0u : off < 0 ? (1u << -off) - 1 : 0u;
        if (mask && off > -32 && off < n) {
            uint32_t m;
            if (off < 0) {
                m = mask[0] << -off;
            } else {
                const int32_t w = off >> 5;
                const uint32_t lo = mask[w];
                const uint32_t hi = w + 1 < words ? mask[w + 1] : 0u;
                m = __funnelshift_r(lo, hi, off & 31);
            }
            const int32_t left = n - off;  // nodes from here on
            bits |= left >= 32 ? m : m & ((1u << left) - 1);
        }
        vis[i] = bits;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (missing >> k & 1)
            vis[k >> 1] &= ~(0xffffu << (16 * (k & 1)));
    return make_uint2(vis[0], vis[1]);
}

// Adds the values of the nodes in `bad`, which the products left out, to features
// [f0, f0 + 16) of a row's O (relative to 2^(N + D)).
template <int D, bool F8>
__device__ __noinline__ void add_apart(const TreeParams& p, int32_t b, int32_t h, int32_t len,
                                       int32_t n, const uint32_t* bad, const uint32_t* mask,
                                       int32_t gh, int32_t tq, float N, float Dd, int f0, float* o)
{
    const __nv_bfloat16* q = (const __nv_bfloat16*)p.q.p + b * p.q.sb +
                             (int64_t)(h * p.G + gh) * p.q.sh + (int64_t)tq * p.q.sl;
#pragma unroll 1
    for (int32_t u = 0; u < n; ++u) {
        if (!(bad[u >> 5] & mask[u >> 5] & (1u << (u & 31))))
            continue;
        const int32_t j = len - n + u;
        const int32_t id = page_of(p.c, b, j >> p.c.page_log2);
        if (id < 0)
            continue;
        const int64_t at = (int64_t)id * p.c.page_stride +
                           (((int64_t)h << p.c.page_log2) + (j & (p.c.page - 1))) * D;
        auto cell = [&](const void* cells, int f) {
            return F8 ? e4m3x2_float2(((const uint8_t*)cells)[at + f]).x
                      : __bfloat162float(((const __nv_bfloat16*)cells)[at + f]);
        };
        float dot = 0.f, lu = 0.f;
#pragma unroll 1
        for (int f = 0; f < D; ++f)
            dot = fmaf(__bfloat162float(q[f]), cell(p.c.k, f), dot);
        float x = __fmul_rn(dot, p.scale_log2);
        if (F8) {
            x = __fmul_rn(x, p.c.k_scale[(int64_t)id * p.c.Hkv + h]);
            lu = log2f(p.c.v_scale[(int64_t)id * p.c.Hkv + h]);
        }
        const float w = ex2((x - N) + (lu - Dd));
#pragma unroll 1
        for (int f = 0; f < 16; ++f)
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

// Zeros a row of a V tile if it is not the sequence's or its page is missing, and if it is
// the tree's and has values that are not finite, which it notes.
template <int D, bool F8>
__device__ __noinline__ void mend_values(uint32_t vt, int32_t row, int32_t node, bool gone,
                                         uint32_t* bad_nodes, uint32_t* any_bad)
{
    if (!gone && node < 0)
        return;
    bool bad = false;
    if (!gone) {
        constexpr uint32_t kHi = F8 ? 0x7c000000u : 0x7f800000u, kLo = F8 ? 0x7c00u : 0x7f80u;
#pragma unroll 4
        for (int c = 0; c < D / 8; ++c) {
            const uint4 x = lds128(vt + (c >> 3) * (kTile * 128) + sw128_offset(row, c & 7));
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                bad |= (w[i] & kHi) == kHi || (w[i] & kLo) == kLo;
        }
        if (bad) {
            atomicOr(bad_nodes + (node >> 5), 1u << (node & 31));
            *any_bad = 1;
        }
    }
    if (gone || bad) {
#pragma unroll 4
        for (int c = 0; c < D / 8; ++c)
            st_shared_v4(vt + (c >> 3) * (kTile * 128) + sw128_offset(row, c & 7), 0, 0, 0, 0);
        fence_proxy_async_smem();
    }
}

// A row's factor times a page's key scale.  A row of zeros over a page of zeros would have 0
// here (2^-217), and hidden scores, which are -inf before they are scaled, would become
// NaN: fp32's smallest normal number does as well, since a row times a key is below 2^32.
__device__ __forceinline__ float score_factor(float factor, float scale)
{
    const float f = factor * scale;
    return f < FLT_MIN ? FLT_MIN : f;
}

__device__ __forceinline__ void hide16(uint32_t (&r)[16], uint32_t seen)
{
#pragma unroll
    for (int j = 0; j < 16; ++j)
        r[j] = seen >> j & 1 ? r[j] : 0xff800000u;  // -inf
}

// The weights y of 16 keys as the products' operand, in place of their scores (TMEM): 8
// columns for 16 keys, one behind the other (kColumns: 8, and 8 of second terms, where
// the keys' scores were).  kLanes: `second` rows have second terms alone; kThree: they and
// zeros, the others third terms beside the first.
template <bool F8, Terms TERMS>
__device__ __forceinline__ void store_weights(uint32_t tP, int k, const float (&y)[16], bool second)
{
    uint32_t hi[16];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float a = y[2 * j], b = y[2 * j + 1];
        hi[j] = F8 ? pack_half2(a, b) : pack_bf16x2(a, b);
    }
    // what a term of bf16 (fp16) leaves
    auto rest = [](float& a, float& b, uint32_t term) {
        if (F8) {
            const float2 z = __half22float2(*reinterpret_cast<const __half2*>(&term));
            a -= z.x, b -= z.y;
        } else {
            const uint32_t na = (term << 16) ^ 0x80000000u;
            const uint32_t nb = (term & 0xffff0000u) ^ 0x80000000u;
            f2unpack(f2add(f2pack(a, b), f2pack(__uint_as_float(na), __uint_as_float(nb))), a, b);
        }
    };
    if (by_columns(TERMS) || (TERMS == kLanes && second)) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float a = y[2 * j], b = y[2 * j + 1];
            rest(a, b, hi[j]);
            const uint32_t next = F8 ? pack_half2(a, b) : pack_bf16x2(a, b);
            if (TERMS != kThree) {
                hi[TERMS == kLanes ? j : 8 + j] = next;
            } else if (second) {
                hi[j] = next;
                hi[8 + j] = 0;
            } else {
                rest(a, b, next);
                hi[8 + j] = pack_bf16x2(a, b);
            }
        }
    }
    if (by_columns(TERMS))
        tmem_st16(tP + 16 * k, hi);
    else
        tmem_st8(tP + 8 * k, hi);
}

// Weights of a row's 64 keys from their scores r.  Returns the sum of the terms.
template <bool F8, Terms TERMS, typename INFO>
__device__ __forceinline__ float weights(const uint32_t (&r)[chunks(TERMS)][16], uint32_t tP,
                                         const INFO& ti, int k0, int page_log2, float factor,
                                         float N, float Dd, bool second)
{
    const uint64_t off = f2pack(-N, -N);
    uint64_t sum[2] = {f2pack(0.f, 0.f), f2pack(0.f, 0.f)};
#pragma unroll
    for (int k = 0; k < chunks(TERMS); ++k) {
        float2 sc = make_float2(1.f, 0.f);
        if (F8)
            sc = ti.scale[(k0 + 16 * k) >> page_log2];
        const float fk = F8 ? score_factor(factor, sc.x) : factor, up = F8 ? ex2(sc.y - Dd) : 1.f;
        const uint64_t f2 = f2pack(fk, fk), up2 = f2pack(up, up);
        float y[16];
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
            float a, b;
            f2unpack(f2fma(f2pack(__uint_as_float(r[k][j]), __uint_as_float(r[k][j + 1])), f2, off),
                     a, b);
            uint64_t e = f2pack(ex2(a), ex2(b));
            sum[j >> 1 & 1] = f2add(sum[j >> 1 & 1], e);
            if (F8)
                e = f2mul(e, up2);
            f2unpack(e, y[j], y[j + 1]);
        }
        store_weights<F8, TERMS>(tP, k, y, second);
    }
    float s0, s1, s2, s3;
    f2unpack(sum[0], s0, s1);
    f2unpack(sum[1], s2, s3);
    return (s0 + s1) + (s2 + s3);
}

// The same where scores are far from zero, or the tile's value scales from one another or
// from D: scores are rounded before N is taken off, and weights are powers of their own.
template <bool F8, Terms TERMS, typename INFO>
__device__ __noinline__ float weights_far(uint32_t tS, uint32_t tP, const INFO& ti, int k0,
                                          int page_log2, uint32_t vis0, uint32_t vis1,
                                          float factor, float N, float Dd, bool second)
{
    // (differences in place of all scores first: second terms take the place of some)
    float sum = 0.f;
    uint32_t r[16];
#pragma unroll 1
    for (int k = 0; k < chunks(TERMS); ++k) {
        tmem_ld16(tS + 16 * k, r);
        tmem_ld_wait();
        tmem_reg_fence16(r);
        hide16(r, (k < 2 ? vis0 : vis1) >> (16 * (k & 1)));
        const float fk =
            F8 ? score_factor(factor, ti.scale[(k0 + 16 * k) >> page_log2].x) : factor;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            // (a packed product and sum would be joined to one operation)
            const float x = __fadd_rn(__fmul_rn(__uint_as_float(r[j]), fk), -N);
            sum += ex2(x);
            r[j] = __float_as_uint(x);
        }
        tmem_st16(tS + 16 * k, r);
    }
    tmem_st_wait();
#pragma unroll 1
    for (int k = 0; k < chunks(TERMS); ++k) {
        tmem_ld16(tS + 16 * k, r);
        tmem_ld_wait();
        tmem_reg_fence16(r);
        const float lu = F8 ? ti.scale[(k0 + 16 * k) >> page_log2].y - Dd : 0.f;
        float y[16];
#pragma unroll
        for (int j = 0; j < 16; ++j)
            y[j] = ex2(__uint_as_float(r[j]) + lu);
        store_weights<F8, TERMS>(tP, k, y, second);
    }
    return sum;
}

// A row of a group's O (TMEM) added to what is set apart of it, f times that; f = 0: none.
template <int D>
__device__ __noinline__ void set_apart(uint32_t tO, float4* apart, float f)
{
    tmem_st_wait();
#pragma unroll 1
    for (int c0 = 0; c0 < D; c0 += 32) {
        uint32_t o[32];
        tmem_ld32(tO + c0, o);
        tmem_ld_wait();
        tmem_reg_fence32(o);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            float4* at = apart + (c0 / 4 + k) * kTreeRows;
            float4 x = make_float4(__uint_as_float(o[4 * k]), __uint_as_float(o[4 * k + 1]),
                                   __uint_as_float(o[4 * k + 2]), __uint_as_float(o[4 * k + 3]));
            if (f != 0.f) {
                const float4 y = *at;
                x = make_float4(fmaf(f, y.x, x.x), fmaf(f, y.y, x.y), fmaf(f, y.z, x.z),
                                fmaf(f, y.w, x.w));
            }
            *at = x;
        }
    }
}

// And f times what is set apart added to O.
template <int D>
__device__ __noinline__ void take_back(uint32_t tO, const float4* apart, float f)
{
#pragma unroll 1
    for (int c0 = 0; c0 < D; c0 += 32) {
        uint32_t o[32];
        tmem_ld32(tO + c0, o);
        tmem_ld_wait();
        tmem_reg_fence32(o);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float4 y = apart[(c0 / 4 + k) * kTreeRows];
            o[4 * k] = __float_as_uint(fmaf(f, y.x, __uint_as_float(o[4 * k])));
            o[4 * k + 1] = __float_as_uint(fmaf(f, y.y, __uint_as_float(o[4 * k + 1])));
            o[4 * k + 2] = __float_as_uint(fmaf(f, y.z, __uint_as_float(o[4 * k + 2])));
            o[4 * k + 3] = __float_as_uint(fmaf(f, y.w, __uint_as_float(o[4 * k + 3])));
        }
        tmem_st32(tO + c0, o);
    }
    tmem_st_wait();
}

template <int D, bool F8, Terms TERMS, bool LONG>
__device__ __forceinline__ void softmax(const TreeParams& p, Shared<D, F8>& sh, uint32_t smem,
                                        const WaitCtx& wctx)
{
    using C = Cfg<D, F8>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kChunks = chunks(TERMS);
    const int w = warp >> 2, rit = (warp & 3) * 32 + lane;  // group, row
    const bool second = by_rows(TERMS) && (warp & 2);
    const int half = TERMS == kSplit && second;             // the second of its group's keys
    const int k0 = w * 64 + half * 32;                      // its first key of a tile
    const int row = by_rows(TERMS) ? rit & 63 : rit;       // ..., of the segment
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = lanes + w * 64, tO = lanes + C::kO0;  // (all of TMEM is the block's)
    const int32_t R = p.G * p.T, chain = chain_mask<F8, TERMS, LONG>(p);
    float4* const apart = reinterpret_cast<float4*>(p.apart) +
                          (2 * (int64_t)blockIdx.x + w) * (kTreeRows * D / 4) + rit;
    uint32_t gt = 0, met = 0;
    Ring<C::kS> sr, last;  // the tile's S, and the one before's
    int4 info = make_int4(0, 0, 0, 0);
    Piece run;
    for (uint32_t seg = 0; next_run(sh, seg, run, wctx, 30); ++seg) {
        if (seg == 0) {
            copy_queries<D, F8, TERMS, 8>(p, sh, smem, run, 0, warp);
            if (lane == 0)
                mbar_arrive(&sh.q_first);
        }
        int32_t gh, tq;
        split_row(p, run.rg * kTreeRows + row, gh, tq);
        const bool valid = run.rg * kTreeRows + row < R && tq < run.n;
        const uint32_t* mask =
            valid ? p.mask + ((int64_t)run.b * p.T + tq) * p.words : nullptr;
        float factor = p.scale_log2;
        if (F8) {
            const bool ok = wait(&sh.q_full[seg & 1], (seg >> 1) & 1, wctx, 31) &&
                            (seg > 0 || wait(&sh.q_first, 0, wctx, 31));
            if (!__all_sync(0xffffffffu, ok))
                return;
            factor = sh.qf[seg & 1][rit];
            __syncwarp();
            if (!by_rows(TERMS) && lane == 0)
                mbar_arrive(&sh.q_empty[seg & 1]);
        }
        float N = kNone, Dd = 0.f, l = 0.f;
        for (int32_t i = 0; i < run.nt; ++i, ++gt) {
            const int32_t base = (run.tile0 + i) * kTile + w * 64;  // the group's 64 keys
            bool ok = wait(&sh.info_full[gt % kRing], (gt / kRing) & 1, wctx, 32);
            if (!__all_sync(0xffffffffu, ok))
                return;
            const TileInfo<F8>& ti = sh.info[gt % kRing];
            const uint32_t flags = ti.flags;
            // 16 keys a bit
            uint32_t missing = 0;
            if (flags & 0xffu)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    missing |= (flags >> ((w * 64 + 16 * k) >> p.c.page_log2) & 1u) << k;
            const bool masked = base + 64 > run.len - run.n || missing;
            uint32_t vis[2] = {~0u, ~0u};
            if (masked) {
                const uint2 v = visible(run.len - run.n, run.n, p.words, base, mask, missing);
                vis[0] = v.x, vis[1] = v.y;
            }
            const uint32_t buf = sr.at * 128;
            ok = wait(&sh.s_full[sr.at], sr.phase, wctx, 33);
            if (!__all_sync(0xffffffffu, ok))
                return;
            tc_fence_after();
            float top[kChunks];  // of 16 keys each
            uint32_t r[kChunks][16];
            const uint32_t tR = tS + buf + half * 32, tP = tS + buf + half * 16;
#pragma unroll
            for (int k = 0; k < kChunks; ++k)
                tmem_ld16(tR + 16 * k, r[k]);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < kChunks; ++k)
                tmem_reg_fence16(r[k]);
            if (__builtin_expect(masked, 0)) {
                if (half)
                    vis[0] = vis[1];
#pragma unroll
                for (int k = 0; k < kChunks; ++k)
                    hide16(r[k], vis[k >> 1] >> (16 * (k & 1)));
            }
#pragma unroll
            for (int k = 0; k < kChunks; ++k) {
                float m = fmaxf(__uint_as_float(r[k][0]), __uint_as_float(r[k][1]));
#pragma unroll
                for (int j = 2; j < 16; j += 2)
                    m = fmax3(m, __uint_as_float(r[k][j]), __uint_as_float(r[k][j + 1]));
                // (rounded: N may become one of them, and is taken off them)
                top[k] = __fmul_rn(
                    m, F8 ? score_factor(factor, ti.scale[(k0 + 16 * k) >> p.c.page_log2].x)
                          : factor);
            }
            const float mx = kChunks == 2 ? fmaxf(top[0], top[1])
                                          : fmaxf(fmax3(top[0], top[1], top[kChunks - 2]),
                                                  top[kChunks - 1]);
            // N up to the largest score, D up to the largest exponent, O with them
            float f = 1.f;
            bool rise = valid && mx - N > grow(F8);
            if (rise) {
                f = ex2(N - mx);
                l *= f;
                Dd += N - mx;
                N = mx;
            }
            if (F8) {
                float me = -INFINITY;
#pragma unroll
                for (int k = 0; k < kChunks; ++k)
                    me = fmaxf(me, (top[k] - N) + ti.scale[(k0 + 16 * k) >> p.c.page_log2].y);
                rise = valid && me - Dd > kTop;
                f = 1.f;
                if (rise) {
                    f = ex2(Dd - (me - head(TERMS)));
                    Dd = me - head(TERMS);
                }
            }
            const bool away = (fabsf(N) >= kFar && N != kNone) || (F8 && Dd < kLow);
            const bool far =
                __any_sync(0xffffffffu, valid && away) || (F8 && (flags & kWideTile));
            if (__builtin_expect(far, 0))
                l += weights_far<F8, TERMS>(tR, tP, ti, k0, p.c.page_log2, vis[0], vis[1], factor,
                                            N, Dd, second);
            else
                l += weights<F8, TERMS>(r, tP, ti, k0, p.c.page_log2, factor, N, Dd, second);
            if (TERMS == kSplit) {  // the other half's keys (whose scores nobody reads any more)
                const uint32_t zero[16] = {};
                tmem_st16(tS + buf + (1 - half) * 16, zero);
            }
            const bool end_chain = i > 0 && (i & chain) == 0;
            const bool rises = __any_sync(0xffffffffu, rise);
            if (i > 0 && (rises || end_chain)) {
                // (late, since it has to wait for the product before this one)
                ok = wait(&sh.s_free[last.at], last.phase, wctx, 37);
                if (!__all_sync(0xffffffffu, ok))
                    return;
                tc_fence_after();
#pragma unroll 1
                for (int c0 = 0; c0 < (rises ? D : 0); c0 += 32) {
                    uint32_t o[32];
                    tmem_ld32(tO + w * D + c0, o);
                    tmem_ld_wait();
                    tmem_reg_fence32(o);
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                    tmem_st32(tO + w * D + c0, o);
                }
                if (i > chain)
                    sh.n[w][rit] *= f;
                if (end_chain) {
                    set_apart<D>(tO + w * D, apart, i > chain + 1 ? sh.n[w][rit] : 0.f);
                    sh.n[w][rit] = 1.f;
                }
            }
            tmem_st_wait();
            if (masked) {  // V's rows that not everyone sees
                const uint32_t vs = gt % C::kV;
                ok = wait(&sh.v_full[vs], (gt / C::kV) & 1, wctx, 34);
                if (!__all_sync(0xffffffffu, ok))
                    return;
                if (rit < 64) {
                    const int32_t j = base + rit;
                    mend_values<D, F8>(smem + C::kV0 + vs * C::kTileBytes, w * 64 + rit,
                                       j - (run.len - run.n),
                                       j >= run.len || (missing >> (rit >> 4) & 1),
                                       sh.bad[seg % 3], &sh.any_bad[seg % 3]);
                }
            }
            tc_fence_before();
            mbar_arrive(&sh.p_full[w][sr.at]);
            last = sr;
            sr.next();
        }
        // ---- the segment's rows.  (When its last product is done, nobody reads the groups'
        // sums of the segment before any more.)
        bool ok = wait(&sh.s_free[last.at], last.phase, wctx, 35);
        if (!__all_sync(0xffffffffu, ok))
            return;
        if (run.nt - 1 > chain) {
            tc_fence_after();
            take_back<D>(tO + w * D, apart, sh.n[w][rit]);
            tc_fence_before();
        }
        sh.n[w][rit] = N;
        sh.l[w][rit] = l;
        if (F8)
            sh.d[w][rit] = Dd;
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&sh.meet);
        ok = wait(&sh.meet, met, wctx, 36);
        met ^= 1;
        if (!__all_sync(0xffffffffu, ok))
            return;
        tc_fence_after();
        if (threadIdx.x < 32) {  // for the segment after the next (see `bad`)
            sh.bad[(seg + 2) % 3][lane] = 0;
            if (lane == 0)
                sh.any_bad[(seg + 2) % 3] = 0;
        }
        const float na = sh.n[0][rit], nb = sh.n[1][rit];
        const float nc = TERMS == kSplit ? sh.n[0][rit ^ 64] : na;
        const float nd = TERMS == kSplit ? sh.n[1][rit ^ 64] : nb;
        const float nx = TERMS == kSplit ? fmaxf(fmaxf(na, nb), fmaxf(nc, nd)) : fmaxf(na, nb);
        float da = na - nx, db = nb - nx, dx = 0.f;
        l = sh.l[0][rit] * ex2(da) + sh.l[1][rit] * ex2(db);
        if (TERMS == kSplit)
            l += sh.l[0][rit ^ 64] * ex2(nc - nx) + sh.l[1][rit ^ 64] * ex2(nd - nx);
        if (F8) {
            da += sh.d[0][rit];
            db += sh.d[1][rit];
            dx = fmaxf(da, db);
            if (TERMS == kSplit)
                dx = fmaxf(dx, fmaxf((nc - nx) + sh.d[0][rit ^ 64], (nd - nx) + sh.d[1][rit ^ 64]));
        }
        const float fa = ex2(da - dx), fb = ex2(db - dx);
        const bool whole = run.nt == run.tiles;
        const int64_t slot = 2 * (int64_t)blockIdx.x + (run.tile0 == 0 ? 1 : 0);
        const int64_t prow = slot * kTreeRows + row;
        // (a partial's O: four features of all rows, then the next four)
        float4* const pout = reinterpret_cast<float4*>(p.part_o) + slot * (kTreeRows * D / 4) + row;
        const int64_t orow =  // (of the segment one behind the other)
            ((int64_t)run.b * p.Hq + run.h * p.G) * p.T + run.rg * kTreeRows + row;
        const float2 inv = row_factors<D, F8>(dx, l);
        // The groups take half of the features each, 16 at a time.  By rows: the two rows of a
        // query hand each other half of those, by way of the segment's queries, which are done
        // with (one row handing over all: 256 short sequences 146 us in place of 139, in 8 bits
        // 195 in place of 182).
        const uint32_t pass = smem + (seg & 1) * C::kTileBytes + w * (64 * D * 2) + row * (D * 2);
        auto chunk = [&](int c, int k) {  // 16 bytes k of 16 features c
            return pass + (((4 * c + k) ^ (row & 7)) << 4);
        };
#pragma unroll 1
        for (int s = 0; s < D / 32; ++s) {
            const int c = by_rows(TERMS) && !second ? s ^ (D / 64) : s;
            const int c0 = w * (D / 2) + 16 * c;
            float o[16];
            uint32_t ta[16], tb[16];
            tmem_ld16(tO + c0, ta);
            tmem_ld16(tO + D + c0, tb);
            tmem_ld_wait();
            tmem_reg_fence16(ta);
            tmem_reg_fence16(tb);
#pragma unroll
            for (int k = 0; k < 16; ++k)
                o[k] = fmaf(fa, __uint_as_float(ta[k]), fb * __uint_as_float(tb[k]));
            if (by_rows(TERMS)) {
                if (s < D / 64) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        st_shared_v4(chunk(c, k), __float_as_uint(o[4 * k]),
                                     __float_as_uint(o[4 * k + 1]), __float_as_uint(o[4 * k + 2]),
                                     __float_as_uint(o[4 * k + 3]));
                    continue;
                }
                if (s == D / 64) {
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&sh.handed);
                    ok = wait(&sh.handed, met ^ 1, wctx, 39);
                    if (!__all_sync(0xffffffffu, ok))
                        return;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint4 x = lds128(chunk(c, k));
                    o[4 * k] += __uint_as_float(x.x), o[4 * k + 1] += __uint_as_float(x.y);
                    o[4 * k + 2] += __uint_as_float(x.z), o[4 * k + 3] += __uint_as_float(x.w);
                }
            }
            if (!valid)
                continue;
            if (__builtin_expect(sh.any_bad[seg % 3], 0)) {
                float y[16];
#pragma unroll
                for (int k = 0; k < 16; ++k)
                    y[k] = o[k];
                add_apart<D, F8>(p, run.b, run.h, run.len, run.n, sh.bad[seg % 3], mask, gh, tq, nx,
                                 dx, c0, y);
#pragma unroll
                for (int k = 0; k < 16; ++k)
                    o[k] = y[k];
            }
            if (whole)
#pragma unroll
                for (int k = 0; k < 16; ++k)
                    o[k] = F8 ? o[k] * inv.x * inv.y : o[k] * inv.x;
            if (!whole || is_fp32<F8, TERMS>(p)) {
                float4* to = whole ? reinterpret_cast<float4*>((float*)p.o + orow * D + c0)
                                   : pout + (c0 / 4) * kTreeRows;
                const int step = whole ? 1 : kTreeRows;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    to[k * step] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
            } else {
                uint4* to = reinterpret_cast<uint4*>((__nv_bfloat16*)p.o + orow * D + c0);
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    to[k] = make_uint4(pack_bf16x2(o[8 * k], o[8 * k + 1]),
                                       pack_bf16x2(o[8 * k + 2], o[8 * k + 3]),
                                       pack_bf16x2(o[8 * k + 4], o[8 * k + 5]),
                                       pack_bf16x2(o[8 * k + 6], o[8 * k + 7]));
            }
        }
        tc_fence_before();
        mbar_arrive(&sh.o_empty);
        if (by_rows(TERMS)) {
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sh.q_empty[seg & 1]);
        }
        if (valid && w == 0 && !second) {
            if (whole)
                p.lse[orow] = row_lse(nx, l);
            else
                p.part_ndl[prow] = make_float4(nx, dx, l, 0.f);
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

// LONG: segments may have more tiles than a chain
template <int D, bool F8, Terms TERMS, bool LONG>
__global__ void __launch_bounds__(Cfg<D, F8>::kThreads, 1)
    decode_tree_kernel(const __grid_constant__ CUtensorMap tk,
                       const __grid_constant__ CUtensorMap tv, const __grid_constant__ TreeParams p)
{
    using C = Cfg<D, F8>;
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_u32(smem) & 1023) {  // (the swizzle patterns begin there)
        if (threadIdx.x == 0) {
            p.info[blockIdx.x] = make_int4(0, 0, 0, 0);
            cache_fault(p.c.status, kSiteShared, blockIdx.x);
        }
        return;
    }
    Shared<D, F8>& sh = *reinterpret_cast<Shared<D, F8>*>(smem + C::kShared0);
    const uint32_t base = smem_u32(smem);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        sh.abort = 0;
        for (int s = 0; s < C::kK; ++s) {
            mbar_init(&sh.k_full[s], F8 ? 4 : 1);
            mbar_init(&sh.k_empty[s], 1);
        }
        for (int s = 0; s < C::kV; ++s) {
            mbar_init(&sh.v_full[s], F8 ? 4 : 1);
            mbar_init(&sh.v_empty[s], 1);
        }
        for (int s = 0; s < C::kRaw; ++s) {
            mbar_init(&sh.raw_full[s], 1);
            mbar_init(&sh.raw_empty[s], 4);
        }
        for (int s = 0; s < C::kS; ++s) {
            mbar_init(&sh.s_full[s], 1);
            mbar_init(&sh.s_free[s], 1);
            mbar_init(&sh.p_full[0][s], 128);
            mbar_init(&sh.p_full[1][s], 128);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sh.q_full[s], 1);
            mbar_init(&sh.q_empty[s], F8 || by_rows(TERMS) ? 9 : 1);
        }
        mbar_init(&sh.o_empty, 256);
        mbar_init(&sh.q_first, 8);
        for (int s = 0; s < kRuns; ++s) {
            mbar_init(&sh.run_full[s], 1);
            mbar_init(&sh.run_empty[s], C::kReaders);
        }
        for (int s = 0; s < kRing; ++s)
            mbar_init(&sh.info_full[s], 1);
        mbar_init(&sh.meet, 8);
        mbar_init(&sh.handed, 8);
        fence_barrier_init();
        prefetch_tmap(&tk);
        prefetch_tmap(&tv);
        p.info[blockIdx.x] = make_int4(0, 0, 0, 0);  // for a block that gives up
    }
    if (warp == 8) {
        tmem_alloc(&sh.tmem, 512);
        tmem_relinquish();
    }
    find_range<C::kThreads>(p, sh);
    if (threadIdx.x < 96)
        sh.bad[threadIdx.x / 32][threadIdx.x % 32] = 0;
    if (threadIdx.x < 3)
        sh.any_bad[threadIdx.x] = 0;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const WaitCtx wctx{&sh.abort, p.c.status, p.timeout_ns};
    if (sh.tmem != 0) {  // (all 512 columns: they begin at 0)
        if (threadIdx.x == 0)
            cache_fault(p.c.status, kSiteShared, blockIdx.x);
    } else if (warp < 8) {
        softmax<D, F8, TERMS, LONG>(p, sh, base, wctx);
    } else if (warp == 8) {
        multiply_scores<D, F8>(sh, base, wctx);
    } else if (warp == 10) {
        multiply_values<D, F8, TERMS>(sh, base, chain_mask<F8, TERMS, LONG>(p), wctx);
    } else if (warp == 9) {
        produce<D, F8>(p, sh, base, tk, tv, wctx);
        if (*wctx.abort_flag) {
            // let copies in flight land before the block's shared memory goes
            const uint64_t t0 = globaltimer_ns();
            while (globaltimer_ns() - t0 < 2000000ull) {
            }
        }
    } else if (warp < 12) {
        load_queries<D, F8, TERMS>(p, sh, base, wctx);
    } else if constexpr (F8) {
        convert<D>(sh, base, wctx);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(sh.tmem, 512);
    }
}

// Rows of the segments that several blocks share: block c holds such a segment's
// beginning, the info[c].z blocks of its group after it the rest.  A block takes 32 rows'
// 32 features, a thread four of a row: a warp reads four features of all rows, as they lie
// together, and the rows are put together again in shared memory.
template <int D, bool F8>
__global__ void __launch_bounds__(256) merge_kernel(const __grid_constant__ TreeParams p)
{
    constexpr int kAtOnce = 4;  // partials on their way
    __shared__ float4 out[32][9];
    const int4 info = p.info[blockIdx.x];
    const int k = info.z + 1;
    const int32_t h = info.y / p.row_groups, r0 = (info.y - h * p.row_groups) * kTreeRows;
    const int32_t first = blockIdx.y / (D / 32) * 32;  // row of the block's first
    if (info.z <= 0 || r0 + first >= p.G * p.T)
        return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.y % (D / 32) * 8;           // the block's features, by four
    const int own = 2 * blockIdx.x, step = 2 * p.row_groups;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float nx = kNone, dx = F8 ? -INFINITY : 0.f, L = 0.f;
    const float4* parts = reinterpret_cast<const float4*>(p.part_o) + first + lane;
    for (int i0 = 0; i0 < k; i0 += kAtOnce) {
        float4 y[kAtOnce], o[kAtOnce];  // reference, exponent and sum; O
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const int64_t slot = i0 + j == 0 ? own + 1 : own + (i0 + j) * step;
            y[j] = make_float4(kNone, F8 ? -INFINITY : 0.f, 0.f, 0.f);
            o[j] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i0 + j < k) {
                y[j] = p.part_ndl[slot * kTreeRows + first + lane];
                o[j] = parts[(slot * (D / 4) + c + warp) * kTreeRows];
            }
        }
        float n2 = nx;
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j)
            n2 = fmaxf(n2, y[j].x);
        float d2 = dx;
        if (F8) {
            d2 += nx - n2;
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j)
                d2 = fmaxf(d2, (y[j].x - n2) + y[j].y);
        }
        const float down = i0 == 0 ? 0.f : ex2((nx - n2) + (F8 ? dx - d2 : 0.f));
        acc.x *= down, acc.y *= down, acc.z *= down, acc.w *= down;
        L *= ex2(nx - n2);
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            if (i0 + j >= k)
                break;
            const float w = ex2((y[j].x - n2) + (F8 ? y[j].y - d2 : 0.f));
            L = fmaf(y[j].z, ex2(y[j].x - n2), L);
            acc.x = fmaf(w, o[j].x, acc.x), acc.y = fmaf(w, o[j].y, acc.y);
            acc.z = fmaf(w, o[j].z, acc.z), acc.w = fmaf(w, o[j].w, acc.w);
        }
        nx = n2;
        dx = d2;
    }
    const float2 inv = row_factors<D, F8>(dx, L);
    if (F8)
        acc.x *= inv.x, acc.y *= inv.x, acc.z *= inv.x, acc.w *= inv.x;
    const float last = F8 ? inv.y : inv.x;
    out[lane][warp] = make_float4(acc.x * last, acc.y * last, acc.z * last, acc.w * last);
    __syncthreads();
    int32_t gh, tq;
    if (c == 0 && warp == 0 && r0 + first + lane < p.G * p.T) {
        split_row(p, r0 + first + lane, gh, tq);
        if (tq < info.w)
            p.lse[((int64_t)info.x * p.Hq + h * p.G + gh) * p.T + tq] = row_lse(nx, L);
    }
    const int r = threadIdx.x >> 3, f = threadIdx.x & 7;
    if (r0 + first + r >= p.G * p.T)
        return;
    split_row(p, r0 + first + r, gh, tq);
    if (tq >= info.w)
        return;
    const float4 x = out[r][f];
    const int64_t at = (((int64_t)info.x * p.Hq + h * p.G + gh) * p.T + tq) * D + (c + f) * 4;
    if (p.o_fp32)
        *reinterpret_cast<float4*>((float*)p.o + at) = x;
    else
        *reinterpret_cast<uint2*>((__nv_bfloat16*)p.o + at) =
            make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
}

template <int D, bool F8, Terms TERMS, bool LONG = true>
cudaError_t launch(const CUtensorMap& tk, const CUtensorMap& tv, TreeParams& p, int num_sms,
                   cudaStream_t stream)
{
    using C = Cfg<D, F8>;
    static_assert(kSmem<D, F8> <= 232448, "shared memory");
    cudaError_t e = cudaFuncSetAttribute(decode_tree_kernel<D, F8, TERMS, LONG>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kSmem<D, F8>);
    if (e != cudaSuccess)
        return e;
    // a block an SM, no more than there can be pieces
    const int64_t segments = (int64_t)p.c.B * p.c.Hkv;  // of one row group
    const int32_t longest = max(1, ceil_div(p.c.max_pages * p.c.page, kTile));
    p.whole = longest <= kWhole;
    const int64_t pieces = min(segments, (int64_t)kTreeMaxCtas) * (p.whole ? 1 : longest);
    p.row_groups = ceil_div(p.G * p.T, kTreeRows);
    const int most = min(kTreeMaxCtas, num_sms);
    p.line_blocks = (int)min((int64_t)max(1, most / p.row_groups), pieces);
    const int grid = p.line_blocks * p.row_groups;
    p.segment_cost = C::segment_cost(p.G * p.T);
    decode_tree_kernel<D, F8, TERMS, LONG>
        <<<grid, C::kThreads, kSmem<D, F8>, stream>>>(tk, tv, p);
    e = cudaGetLastError();
    if (e != cudaSuccess || p.whole)
        return e;
    const int rows = min(kTreeRows, p.G * p.T);
    merge_kernel<D, F8><<<dim3(grid, ceil_div(rows, 32) * (D / 32)), 256, 0, stream>>>(p);
    return cudaGetLastError();
}

template <int D, bool F8>
cudaError_t launch_terms(const CUtensorMap& tk, const CUtensorMap& tv, TreeParams& p, int num_sms,
                         cudaStream_t stream)
{
    // (see "Rounding" above, and is_fp32)
    if constexpr (F8)
        if (!p.o_fp32) {
            const bool many = p.G * p.T > 64;
            if (p.c.max_pages * p.c.page > kLongChain * kTile)
                return many ? launch<D, F8, kOne>(tk, tv, p, num_sms, stream)
                            : launch<D, F8, kSplit>(tk, tv, p, num_sms, stream);
            return many ? launch<D, F8, kOne, false>(tk, tv, p, num_sms, stream)
                        : launch<D, F8, kSplit, false>(tk, tv, p, num_sms, stream);
        }
    if (p.G * p.T > 64)
        return launch<D, F8, kColumns>(tk, tv, p, num_sms, stream);
    if constexpr (!F8)
        if (p.o_fp32)
            return launch<D, F8, kThree>(tk, tv, p, num_sms, stream);
    return launch<D, F8, kLanes>(tk, tv, p, num_sms, stream);
}

}  // namespace tree

cudaError_t launch_decode_tree(const CUtensorMap& tk, const CUtensorMap& tv, TreeParams& p,
                               int num_sms, cudaStream_t stream)
{
    if (p.c.e4m3)
        return p.c.d == 128 ? tree::launch_terms<128, true>(tk, tv, p, num_sms, stream)
                            : tree::launch_terms<64, true>(tk, tv, p, num_sms, stream);
    return p.c.d == 128 ? tree::launch_terms<128, false>(tk, tv, p, num_sms, stream)
                        : tree::launch_terms<64, false>(tk, tv, p, num_sms, stream);
}

}  // namespace dfa
