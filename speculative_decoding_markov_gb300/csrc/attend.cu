// attend.cu - attention of packed windows over a paged key/value cache on the
// tcgen05 tensor cores.
//
// Mathematics.  A row is one query head of one window token; the rows of a
// request that share a kv head (its query heads side by side, token by token)
// share their keys, so they are packed into the 128 lanes of one tile.  Per
// tile of 128 keys, with s = q k^T and x = s * scale * log2 e:
//     m' = max(m, max_j x_j)           l' = l 2^(m - m') + sum_j 2^(x_j - m')
//     o' = o 2^(m - m') + sum_j bf16(2^(x_j - m')) v_j     out = o / l
// m is only moved when a tile exceeds it by more than 2^8 (kLazy): any m near
// the maximum serves, and o, which lives in tensor memory, is then rescaled
// in the first tiles of a row and hardly ever after.
//
// Work.  A block is up to two sub-tiles of one request and kv head, a sub-tile
// the rows of as many whole tokens as 128 lanes hold.  A block larger than one
// sub-tile runs in `pair` form: both softmax warpgroups see every key tile,
// each for its own 128 rows.  A smaller one runs in `stream` form: the
// warpgroups take alternate key tiles of the same rows and their (m, l, o) are
// joined at its end.  The key tiles of all blocks laid end to end are cut into
// shares of equal cost, one per CTA (one CTA per SM, persistent): a long
// context is split over as many SMs as it fills, many short ones share an SM,
// and no schedule is kept between calls.  Blocks that a cut splits leave (m,
// l, o) in the workspace and attend_merge_kernel joins them in the order of
// the keys, so results do not depend on timing.
//
// Pipeline of a CTA: one warp walks the share and hands each block to the
// others; a producer brings K and V tiles page by page with TMA into a ring;
// one brings Q and clears values (below); one issues S = Q K^T and O += P V;
// eight do the softmax, S from tensor memory to registers and P back over S;
// e4m3: a warpgroup each turns K's and V's codes into bf16, exactly, the scale
// included, in a second ring.  Each softmax warpgroup's S, P and O are its
// own, so one's softmax runs beside the other's products.
//
// What bounds it (32 query heads on 8 kv heads of 128, bf16, unless said; times
// of whole calls among others of their kind, merge included):
//   64 windows of 1 to 8 tokens over 300 to 8000: HBM, 5.8 TB/s (105 us).
//   A prompt of 8192 tokens: the softmax between its two products, 1.26
//   PFLOP/s (435 us; this kernel by itself 419, tensor pipe 56 %).  A 128 x 128 tile's softmax takes 1112
//   clocks alone and 1800 beside the other warpgroup's, its two products with
//   their hand-overs 1460; S has no room for a second buffer beside O.
//   e4m3 windows: turning the codes into bf16, about 5700 warp instructions a
//   tile of 128 keys and 50 % of the issue slots: 3.4 TB/s of codes at two
//   contexts of 150001 to 199999 (28 heads on 4, 102 us).
//   One token over 500 keys: the chain of plan, loads, two products and merge
//   (12.5 us, 12.0 in a graph).
// The warps' loops together have to stay in the instruction cache: unrolling
// one of them twice more than now cost 5 to 40 %, wherever it was tried.
//
// What a row does not see does not reach it: scores are replaced, not added
// to; values of a tile that some row sees only in part are cleared of NaN and
// infinities in shared memory, and the rows that do see one get its product
// from add_nonfinite() at the end.
#include <cudaTypedefs.h>

#include <algorithm>

#include "paged.cuh"

namespace sdm {
namespace {

constexpr int kTile = 128;            // keys per tile, rows per sub-tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLazy = 8.0f;
// The running maximum stays finite, so that the weight of an infinite score is
// infinite (not 2^(inf - inf)) and the row's log-sum-exp with it.
constexpr float kMaxRef = 3.0e38f;
// The weights enter the second product as bf16: an error of at most 2^-8 of a
// weight, which the sum over many keys that count averages out.  Where a row
// sees few keys it does not, so the remainder p - bf16(p) is multiplied too: in
// blocks of at most kStackTiles key tiles that leave half of the 128 lanes free
// as rows of the same product (row r in lane r of its 16, the remainder 16
// lanes on), in blocks of at most kFineTiles by a second one.  The limits weigh
// cost against length: a row over more keys of which few count has the
// weights' error in full.  Largest error on peaked rows (scores of deviation 8
// to 11), in units of 2^-8 sum p |v|, of which rounding the result is 1: with
// the remainders 0.91 to 1.00; without, 1.24 over 2049 keys, 1.24 over 2500,
// 1.18 over 40000.
// Cost against no remainders at all: 256 e4m3 windows over 200 to 4000 tokens
// 137 -> 149 us, five e4m3 windows of 37 to 1500 tokens 57 -> 67 us, 32 trees
// of 65 slots 132 -> 134 us, a prompt of 8192 430 -> 435 us, one token over 500
// keys 12.0 -> 12.5 us.
constexpr int kStackRows = 64;
constexpr int kFineTiles = 9, kStackTiles = 16;
constexpr int kTmemCols = 512;        // S0, S1, O0, O1 at columns 0, 128, 256, 384; P over S

// One block, as the walking warp hands it to the others.
struct Blk {
    int i, hk, row0, n;               // request, kv head, first packed row and rows of its window
    int ctx, m0, M, p1;               // committed tokens; first row and rows of the block, its last window position
    int ns, lo, tiles, t0;            // Geom's; the share's key tiles of the block are t0 .. t1 - 1
    int t1, flags, p0, nonfinite;     // t1 = 0: no more blocks; set if a cleared value was not finite
};
enum { BLK_PAIR = 1, BLK_STACKED = 2, BLK_TWICE = 4 };

// SMALL: all windows of the call fit in kStackRows rows.  Their calls are
// bound by loads, and the second sub-tile of Q that they do not need holds two
// more tiles of the rings: 64 windows of 1 to 8 tokens 105 us against 119, 256
// e4m3 windows 149 against 183, two e4m3 contexts of 150001 to 199999 102
// against 143, one token over 500 keys 12.5 against 12.9.
template <int D, bool E4M3, bool SMALL>
struct Cfg {
    static constexpr int kThreads = E4M3 ? 640 : 384;
    // registers of a thread: the softmax warpgroups', the others' (together
    // the launch's own: 5 x 96 and 3 x 168)
    static constexpr int kRegsSoft = E4M3 ? 144 : 208, kRegsRest = E4M3 ? 64 : 88;
    static_assert(E4M3 ? 2 * kRegsSoft + 3 * kRegsRest == 5 * 96 : 2 * kRegsSoft + kRegsRest == 3 * 168, "registers");
    static constexpr int kQBytes = kTile * D * 2;            // one 128-row sub-tile
    static constexpr int kTileBytes = kTile * D * 2;         // one bf16 K or V tile
    static constexpr int kQs = SMALL ? 1 : 2;                // sub-tiles of Q
    static constexpr int kRawSlots = !E4M3 ? 0 : D == 64 ? 6 : SMALL ? 4 : 2;
    static constexpr int kFit = (224 * 1024 - kQs * kQBytes - kRawSlots * kTile * D) / kTileBytes;
    static constexpr int kSlots = kFit < 8 ? kFit : 8;
    static constexpr int kRingBlocks = E4M3 && D == 128 && !SMALL ? 3 : 8;   // blocks handed out ahead
    static constexpr int kXchRows = SMALL ? kStackRows : kTile;
    static constexpr int kRawBytes = kTile * D;              // e4m3 codes of a tile
    static constexpr int kRing = kQs * kQBytes;
    static constexpr int kRaw = kRing + kSlots * kTileBytes;
    static constexpr int kExps = kRaw + kRawSlots * kRawBytes;
    static constexpr int kXch = kExps + kRawSlots * kTile;   // (m, l) of both warpgroups' rows
    static constexpr int kBlks = kXch + 2 * kXchRows * 8;
    static constexpr int kBars = kBlks + kRingBlocks * static_cast<int>(sizeof(Blk));
    static constexpr int kNumBars = (E4M3 ? 2 * kSlots + 1 : 3 * kSlots) + 2 * (kRawSlots > 0 ? kRawSlots : 1) +
                                    2 * kRingBlocks + 13;
    static constexpr int kMisc = kBars + kNumBars * 8;
    static constexpr int kTotal = kMisc + 16;
    static_assert(kTotal <= 232448, "shared memory");
    static_assert(kSlots >= 4, "a K tile beside the two V tiles before it");
    // K and V are converted apart: each kind has slots of its own, whose every phase its warps wait for
    static_assert(!E4M3 || (kSlots % 2 == 0 && kRawSlots % 2 == 0), "slots of a kind");
};

struct Share {             // per CTA, for the merge: the block its last segment starts, and how its first goes on
    int rows;              // rows of the block that its last segment starts and does not finish; 0: none
    int row0, m0, hk;      // that block: first packed row of its window, first row, kv head
    int head;              // its first segment continues a block: 0 no, 1 and finishes it, 2 and does not; 3: no work
    int pad[3];
};

struct Scratch {
    Share* share;          // [grid]
    float2* ml;            // [2 grid][cap]: (m, l) of split blocks' rows
    float* o;              // [2 grid][cap][D]
    int cap;               // rows per slot
};

// ---------------------------------------------------------------------------
// Geometry: a request's blocks, a block's key tiles, a CTA's share of them
// ---------------------------------------------------------------------------
struct Geom {
    int m0, M;             // first row and rows of the block
    int p0, p1;            // window positions of its first and last row
    int ns, lo, n;         // tiles 0 .. ns - 1 hold the sinks, tiles ns .. n - 1 are key tiles lo, lo + 1, ...
    bool pair;             // two sub-tiles
    int weight;            // cost of a key tile, in units of the shares
    // how the weights' rounding to bf16 is made up for where there are few keys
    bool stacked;          // their remainders are more rows of the same product
    bool twice;            // their remainders are multiplied in a second product
};

__device__ __forceinline__ int blocks_of(const AttendParams& p, const Window& w) {
    return (w.n * p.group + 2 * p.sub - 1) / (2 * p.sub);
}

__device__ __forceinline__ Geom geom_of(const AttendParams& p, const Window& w, int b) {
    Geom g;
    g.m0 = b * 2 * p.sub;
    g.M = min(2 * p.sub, w.n * p.group - g.m0);
    g.p0 = g.m0 / p.group;
    g.p1 = (g.m0 + g.M - 1) / p.group;
    const int end = p.tree ? w.ctx + w.n : w.ctx + g.p1 + 1;
    g.ns = g.lo = 0;
    if (p.window > 0) {
        g.lo = max(0, w.ctx + (p.tree ? 0 : g.p0) + 1 - p.window) / kTile;
        g.ns = min((p.sinks + kTile - 1) / kTile, g.lo);
    }
    g.n = g.ns + (end + kTile - 1) / kTile - g.lo;
    g.pair = g.M > p.sub;
    g.stacked = g.M <= kStackRows && g.n <= kStackTiles;
    g.twice = !g.stacked && g.n <= kFineTiles;
    g.weight = g.pair ? (g.twice ? p.cost_twice : p.cost_pair) : p.cost_stream;
    return g;
}

__device__ __forceinline__ int tile_key(const Blk& b, int t) { return (t < b.ns ? t : b.lo + t - b.ns) * kTile; }

// Whether some row at window positions p0 .. p1 does not see all of the tile's keys.
__device__ __forceinline__ bool tile_mixed(const AttendParams& p, int ctx, int p0, int p1, int key0) {
    const int last = key0 + kTile - 1;
    if (last > (p.tree ? ctx - 1 : ctx + p0)) return true;
    if (p.window <= 0 || last < p.sinks) return false;
    // a tree row's depth is what its bits say, those past the window's tokens counted
    return key0 <= ctx + (p.tree ? p.words * 32 - 1 : p1) - p.window;
}

// Whether the tile's values are cleared of NaN and infinities: a row may not
// see them, or a remainder (of either sign) may meet an infinity.
__device__ __forceinline__ bool tile_cleaned(const AttendParams& p, const Blk& b, int key0) {
    return (b.flags & BLK_TWICE) || tile_mixed(p, b.ctx, b.p0, b.p1, key0);
}

struct Start {
    unsigned long long us, u0, u1;   // unit at which the first block begins, the CTA's units [u0, u1)
    int i, b, hk;
};

// How many of a block's n tiles begin before unit u, the first at unit `at`.
__device__ __forceinline__ int tiles_before(unsigned long long u, unsigned long long at, unsigned wt, int n) {
    if (u <= at) return 0;
    const unsigned long long d = u - at;
    if (d >= static_cast<unsigned long long>(n) * wt) return n;
    return static_cast<int>((static_cast<unsigned>(d) + wt - 1) / wt);   // n * wt is below 2^32
}

// Walks the blocks of a CTA's share.
struct Walk {
    unsigned long long us, u0, u1;
    int i, b, hk;
    int have;              // request whose window (and block whose geometry) is loaded
    int have_b;
    Window w;
    Geom g;
    int t0, t1;            // the share's key tiles of the current block

    __device__ __forceinline__ void init(const Start& s) {
        us = s.us;
        u0 = s.u0;
        u1 = s.u1;
        i = s.i;
        b = s.b;
        hk = s.hk - 1;
        have = have_b = -1;
    }

    __device__ __forceinline__ bool next(const AttendParams& p) {
        if (have >= 0) us += p.cost_block + g.n * g.weight;
        for (;;) {
            if (us >= u1) return false;
            if (++hk >= p.c.heads) {
                hk = 0;
                ++b;
            }
            for (;;) {
                if (i >= p.R) return false;
                if (have != i) {
                    w = window_of(p.cu, p.ctx, i, p.rows, p.max_window, table_tokens(p.c));
                    have = i;
                    have_b = -1;
                }
                if (b < blocks_of(p, w)) break;
                ++i;
                b = hk = 0;
            }
            if (have_b != b) {
                g = geom_of(p, w, b);
                have_b = b;
            }
            const unsigned wt = g.weight;
            const unsigned long long at = us + p.cost_block;   // unit of the first tile
            t0 = tiles_before(u0, at, wt, g.n);
            t1 = tiles_before(u1, at, wt, g.n);
            if (t0 < t1) return true;
            us += p.cost_block + g.n * wt;
        }
    }
};

__device__ __forceinline__ unsigned long long shfl_up64(unsigned long long v, int d) {
    return __shfl_up_sync(0xffffffffu, v, d);
}

// The units of a request's blocks, for one kv head.
__device__ __forceinline__ unsigned long long units_of(const AttendParams& p, const Window& w, int b0, int step) {
    unsigned long long c = 0;
    for (int b = b0; b < blocks_of(p, w); b += step) {
        const Geom g = geom_of(p, w, b);
        c += static_cast<unsigned long long>(p.cost_block + g.n * g.weight);
    }
    return c;
}

// The units [u0, u1) of this CTA, of `total`: the first (total mod grid) CTAs
// get one more than the others.
__device__ __forceinline__ void share_of(unsigned long long total, unsigned long long& u0, unsigned long long& u1) {
    const unsigned long long each = total >> 32 ? total / gridDim.x : static_cast<unsigned>(total) / gridDim.x;
    const unsigned more = static_cast<unsigned>(total - each * gridDim.x);
    u0 = each * blockIdx.x + min(blockIdx.x, more);
    u1 = u0 + each + (blockIdx.x < more ? 1 : 0);
}

// The block of request i in which unit u0 lies; `us` is the request's first
// unit.  Run by a whole warp.
__device__ __forceinline__ void locate(const AttendParams& p, const Window& w, int i, unsigned long long us,
                                       unsigned long long u0, Start& st) {
    const int lane = threadIdx.x & 31;
    const int nb = blocks_of(p, w);
    int found = -1;
    unsigned long long step = 1;
    for (int b0 = 0; b0 < nb && found < 0; b0 += 32) {
        const int b = b0 + lane;
        unsigned long long one = 0;
        if (b < nb) {
            const Geom g = geom_of(p, w, b);
            one = static_cast<unsigned long long>(p.cost_block + g.n * g.weight);
        }
        unsigned long long sum = one * p.c.heads;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long v = shfl_up64(sum, o);
            if (lane >= o) sum += v;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, us + sum > u0);
        const int at = hit ? __ffs(hit) - 1 : 31;
        const unsigned long long before = __shfl_sync(0xffffffffu, sum - one * p.c.heads, at);
        const unsigned long long all = __shfl_sync(0xffffffffu, sum, 31);
        step = __shfl_sync(0xffffffffu, one, at);
        if (hit) {
            found = b0 + at;
            us += before;
        } else {
            us += all;
        }
    }
    const unsigned long long into = u0 - us;
    const unsigned long long k = step == 0 ? 0
                                 : (into | step) >> 32 ? into / step
                                                       : static_cast<unsigned>(into) / static_cast<unsigned>(step);
    st.i = i;
    st.b = max(found, 0);
    st.hk = static_cast<int>(k);
    st.us = us + k * step;
}

// Where this CTA's share starts, for at most 32 requests of at most two blocks
// each: by one warp, a lane per request (the walking warp's first steps are on
// the path of the smallest calls, so they are few).
__device__ __forceinline__ void plan_few(const AttendParams& p, Start& st) {
    const int lane = threadIdx.x & 31;
    Window w = {0, 0, 0, 0};
    if (lane < p.R) w = window_of(p.cu, p.ctx, lane, p.rows, p.max_window, table_tokens(p.c));
    if (w.bad && blockIdx.x == 0) set_status(p.dev_status, w.bad);
    const int nb = blocks_of(p, w);
    unsigned c[2] = {0, 0};
#pragma unroll 1
    for (int b = 0; b < nb; ++b) {
        const Geom g = geom_of(p, w, b);
        (b ? c[1] : c[0]) = p.cost_block + g.n * g.weight;
    }
    const unsigned long long mine = static_cast<unsigned long long>(c[0] + c[1]) * p.c.heads;
    unsigned long long sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long v = shfl_up64(sum, o);
        if (lane >= o) sum += v;
    }
    share_of(__shfl_sync(0xffffffffu, sum, 31), st.u0, st.u1);
    const unsigned hit = __ballot_sync(0xffffffffu, sum > st.u0);
    const int k = hit ? __ffs(hit) - 1 : 0;
    const unsigned c0 = __shfl_sync(0xffffffffu, c[0], k), c1 = __shfl_sync(0xffffffffu, c[1], k);
    unsigned long long us = __shfl_sync(0xffffffffu, sum - mine, k);
    const unsigned long long first = static_cast<unsigned long long>(c0) * p.c.heads;
    st.i = k;
    st.b = st.u0 - us >= first ? 1 : 0;
    if (st.b) us += first;
    const unsigned one = st.b ? c1 : c0;
    const unsigned long long into = st.u0 - us;
    st.hk = one == 0 ? 0 : static_cast<int>(into >> 32 ? into / one : static_cast<unsigned>(into) / one);
    st.us = us + static_cast<unsigned long long>(st.hk) * one;
}

// The same by all warps.  cost: shared memory for R entries.
template <int kThreads>
__device__ __forceinline__ void plan(const AttendParams& p, unsigned long long* cost, Start* start,
                                     unsigned long long* wsum) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int kWarps = kThreads / 32;
    const long long tokens = table_tokens(p.c);
    if (p.max_window * p.group <= 8 * p.sub) {
        for (int i = tid; i < p.R; i += kThreads) {
            const Window w = window_of(p.cu, p.ctx, i, p.rows, p.max_window, tokens);
            if (w.bad && blockIdx.x == 0) set_status(p.dev_status, w.bad);
            cost[i] = units_of(p, w, 0, 1) * p.c.heads;
        }
    } else {   // long windows: their blocks a lane each
        for (int i = warp; i < p.R; i += kWarps) {
            const Window w = window_of(p.cu, p.ctx, i, p.rows, p.max_window, tokens);
            if (w.bad && blockIdx.x == 0 && lane == 0) set_status(p.dev_status, w.bad);
            unsigned long long c = units_of(p, w, lane, 32);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
            if (lane == 0) cost[i] = c * p.c.heads;
        }
    }
    __syncthreads();
    const int per = (p.R + kThreads - 1) / kThreads;
    const int a = min(p.R, tid * per), e = min(p.R, a + per);
    unsigned long long mine = 0;
    for (int i = a; i < e; ++i) mine += cost[i];
    unsigned long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long v = shfl_up64(incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    unsigned long long base = incl - mine, total = 0;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
        const unsigned long long v = wsum[k];
        if (k < warp) base += v;
        total += v;
    }
    unsigned long long u0, u1;
    share_of(total, u0, u1);
    if (tid == 0) {
        start->u0 = u0;
        start->u1 = u1;
    }
    if (u0 < u1 && base <= u0 && u0 < base + mine) {
        int i = a;
        for (; i < e - 1 && u0 >= base + cost[i]; ++i) base += cost[i];
        start->i = i;
        start->us = base;
    }
    __syncthreads();
    if (warp == 0 && u0 < u1) {
        const int i = start->i;
        const unsigned long long us = start->us;
        const Window w = window_of(p.cu, p.ctx, i, p.rows, p.max_window, tokens);
        Start st = {};
        __syncwarp();
        locate(p, w, i, us, u0, st);
        if (lane == 0) {
            start->b = st.b;
            start->hk = st.hk;
            start->us = st.us;
        }
    }
    fence_proxy_async_smem();   // `cost` lies where TMA is about to write
    __syncthreads();
}

// ---------------------------------------------------------------------------
// Barriers: every wait is bounded; a wait that runs out records
// SDM_DEV_TIMEOUT and the role winds down.
// ---------------------------------------------------------------------------
// One short loop (the callers' loops have to fit the instruction cache).
__device__ __forceinline__ bool wait_or_fail(const AttendParams& p, uint64_t* bar, uint32_t parity) {
    if (__builtin_expect(__all_sync(0xffffffffu, mbar_try_wait(bar, parity)), 1)) return true;   // one answer a warp
    const uint64_t t0 = globaltimer();
#pragma unroll 1
    do {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    } while (__all_sync(0xffffffffu, globaltimer() - t0 < kWaitLimitNs));
    set_status(p.dev_status, SDM_DEV_TIMEOUT);
    return false;
}

template <int SLOTS, int RAW, int BLOCKS>
struct Bars {
    // a tile arrives at full; one to be cleaned at dirty, and whoever cleans it
    // arrives at full
    uint64_t full[SLOTS], empty[SLOTS];
    uint64_t dirty[RAW > 0 ? 1 : SLOTS];   // e4m3: the conversion cleans
    uint64_t raw_full[RAW > 0 ? RAW : 1], raw_empty[RAW > 0 ? RAW : 1];
    uint64_t blk_full[BLOCKS], blk_empty[BLOCKS];
    uint64_t q_full, q_empty, s_full[2], p_half[2][2], o_full[2], xch, xdone, drain;   // [warpgroup], [warpgroup][half]
};

// Nonzero if one of the two bf16 in x is an infinity or NaN (the exponent
// field 0xff plus one carries into the sign's place).
__device__ __forceinline__ uint32_t nonfinite2(uint32_t x) { return ((x & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }

// 32 bits: which of the keys base .. base + 31 a row sees.
struct RowView {
    int pos, lo;            // keys <= pos (tree: < ctx) and >= lo or < sinks
    int sinks;
    const uint32_t* bits;   // tree: the row's mask words
    int ctx, n, words;
};

__device__ __forceinline__ uint32_t below(int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; }

__device__ __forceinline__ uint32_t seen32(const RowView& r, int base) {
    uint32_t m = below(r.pos + 1 - base) & (~below(r.lo - base) | below(r.sinks - base));
    if (r.bits) {
        const int o = base - r.ctx;
        if (o > -32 && o < r.n) {
            const int k = o >> 5, sh = o & 31;
            const uint32_t a = k >= 0 && k < r.words ? __ldg(r.bits + k) : 0u;
            const uint32_t b = k + 1 < r.words ? __ldg(r.bits + k + 1) : 0u;
            m |= __funnelshift_r(a, b, sh) & below(r.n - o);
        }
    }
    return m;
}

__device__ __forceinline__ RowView row_view(const AttendParams& p, int i, int ctx, int n_rows, int wp) {
    RowView r;
    r.ctx = ctx;
    r.n = n_rows;
    r.words = p.words;
    r.sinks = p.window > 0 ? p.sinks : 0;
    r.bits = nullptr;
    int pos = ctx + wp;
    r.pos = pos;
    if (p.tree) {
        r.bits = p.tree + (static_cast<size_t>(i) * p.nodes + wp) * p.words;
        int n = 0;
        for (int k = 0; k < p.words; ++k) n += __popc(__ldg(r.bits + k));
        pos = ctx + max(0, n - 1);
        r.pos = ctx - 1;
    }
    r.lo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
    return r;
}

// Adds weight * value for the infinite and NaN values that a row sees in its
// block's partly seen tiles (where shared memory holds zeros for them), to 16
// of its output columns: one thread per row, straight from the cache.  The
// weight of such a value changes nothing while it is a positive number, as it
// is for any finite score, so the row's score is computed only for keys that
// are not finite themselves (with a score for each value 1100 tokens whose
// values are all infinite took 115 ms, and the other warps' waits end after 2 s).
template <int D, bool E4M3>
__device__ __noinline__ void add_nonfinite(const AttendParams& p, const Blk& blk, int m, float m_ref, int col0,
                                           float* o) {
    const int wp = m / p.group;
    const RowView r = row_view(p, blk.i, blk.ctx, blk.n, wp);
    const uint16_t* q = p.q + (blk.row0 + wp) * p.q_stride + static_cast<size_t>(blk.hk * p.group + m % p.group) * D;
    // element c of a cache row, as the products take it
    auto value = [&](const uint8_t* pool, float scale, size_t row, int c) {
        if constexpr (E4M3)   // past bf16's range in one case only: past fp32's, too
            return f16x2_to_f32x2(e4m3x2_to_f16x2(pool[row * D + c])).x * scale;
        else
            return bf16_bits_to_float(reinterpret_cast<const uint16_t*>(pool)[row * D + c]);
    };
    // whether 16 bytes of a row may hold an infinity or NaN
    auto odd16 = [&](uint4 x, float scale) {
        if constexpr (E4M3) {
            uint32_t bad = 0;   // bit 7 of a byte: a code of ones but for its sign
            for (const uint32_t u : {x.x, x.y, x.z, x.w}) bad |= (u & 0x7f7f7f7fu) + 0x01010101u;
            return (bad & 0x80808080u) != 0 || scale > 0x1p119f;   // 448 x 2^119 is the largest finite
        } else {
            return (nonfinite2(x.x) | nonfinite2(x.y) | nonfinite2(x.z) | nonfinite2(x.w)) != 0;
        }
    };
    constexpr int kSize = E4M3 ? 1 : 2;
    for (int t = blk.t0; t < blk.t1; ++t) {
        const int key0 = tile_key(blk, t);
        if (!tile_cleaned(p, blk, key0)) continue;
        for (int j = key0; j < min(key0 + kTile, blk.ctx + blk.n); ++j) {
            if (!((seen32(r, j & ~31) >> (j & 31)) & 1u)) continue;
            const int pg = max(page_of(p.c, blk.i, j), 0);
            const size_t row = pool_row(p.c, pg, j) + (static_cast<size_t>(blk.hk) << p.c.page_shift);
            const float vs = E4M3 ? scale_of(p.c.v_exp[row]) : 1.0f;
            const uint4* v16 = reinterpret_cast<const uint4*>(p.c.v + (row * D + col0) * kSize);
            bool odd = odd16(v16[0], vs);
            if constexpr (!E4M3) odd = odd || odd16(v16[1], vs);
            if (!odd) continue;
            const float ks = E4M3 ? scale_of(p.c.k_exp[row]) : 1.0f;
            const uint4* k16 = reinterpret_cast<const uint4*>(p.c.k + row * D * kSize);
            bool key_odd = false;
            for (int c = 0; c < D * kSize / 16; ++c) key_odd |= odd16(k16[c], ks);
            float weight = 1.0f;
            if (key_odd) {
                float s = 0.f;
                for (int d = 0; d < D; ++d) s = fmaf(bf16_bits_to_float(q[d]), value(p.c.k, ks, row, d), s);
                weight = fast_exp2(s * p.scale * kLog2e - m_ref);
            }
            for (int c = 0; c < 16; ++c) {
                const float x = value(p.c.v, vs, row, col0 + c);
                if (!(fabsf(x) < INFINITY)) o[c] += weight * x;
            }
        }
    }
}

// ---------------------------------------------------------------------------
// The kernel
// ---------------------------------------------------------------------------
// volatile: the order they are written in is kept
__device__ __forceinline__ void ffma2(float& x, float& y, float a, float b) {   // (x, y) = (x, y) * a + b
    asm volatile(
        "{\n\t.reg .b64 v, s, t;\n\tmov.b64 v, {%0, %1};\n\tmov.b64 s, {%2, %2};\n\tmov.b64 t, {%3, %3};\n\t"
        "fma.rn.f32x2 v, v, s, t;\n\tmov.b64 {%0, %1}, v;\n\t}"
        : "+f"(x), "+f"(y)
        : "f"(a), "f"(b));
}

__device__ __forceinline__ void fadd2(float& x, float& y, float a, float b) {   // (x, y) += (a, b)
    asm volatile(
        "{\n\t.reg .b64 v, s;\n\tmov.b64 v, {%0, %1};\n\tmov.b64 s, {%2, %3};\n\tadd.rn.f32x2 v, v, s;\n\t"
        "mov.b64 {%0, %1}, v;\n\t}"
        : "+f"(x), "+f"(y)
        : "f"(a), "f"(b));
}

__device__ __forceinline__ float exp2_in_order(float x) {
    float y;
    asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_in_order(float lo, float hi) {
    uint32_t r;
    asm volatile("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// The largest of a row's 128 scores, N * 32 of them in registers at a time.
template <int N>
__device__ __forceinline__ float tile_max(uint32_t tS) {
    float top = -INFINITY;
#pragma unroll 1
    for (int h = 0; h < 4; h += N) {
        uint32_t y[N][32];
#pragma unroll
        for (int c = 0; c < N; ++c) tmem_ld32(tS + (h + c) * 32, y[c]);
        tmem_ld_wait();
        float z[N];
#pragma unroll
        for (int c = 0; c < N; ++c) {
            z[c] = max3(__uint_as_float(y[c][0]), __uint_as_float(y[c][1]), __uint_as_float(y[c][2]));
#pragma unroll
            for (int j = 3; j < 31; j += 2)
                z[c] = max3(z[c], __uint_as_float(y[c][j]), __uint_as_float(y[c][j + 1]));
            top = max3(top, z[c], __uint_as_float(y[c][31]));
        }
    }
    return top;
}

enum { FORM_PLAIN = 0, FORM_STACKED = 1, FORM_TWICE = 2 };

// 32 scores of a row to weights 2^(x sl + neg), their bf16 pairs to tP and
// their sums.  The order is the pipeline's: the exponentials (4 clocks of a
// scheduler each) have the multiply-add of two pairs on and the sum and the
// rounding of the pair before beside them.
template <int FORM>
__device__ __forceinline__ void weights32(uint32_t (&xs)[32], uint32_t tP, float sl, float neg, bool rest,
                                          float (&l)[4], uint32_t (&held)[16]) {
    float(&x)[32] = reinterpret_cast<float(&)[32]>(xs);
    uint32_t w[16];
    ffma2(x[0], x[1], sl, neg);
    ffma2(x[2], x[3], sl, neg);
    x[0] = exp2_in_order(x[0]);
    x[1] = exp2_in_order(x[1]);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        if (i < 14) ffma2(x[2 * i + 4], x[2 * i + 5], sl, neg);
        if (i < 15) {
            x[2 * i + 2] = exp2_in_order(x[2 * i + 2]);
            x[2 * i + 3] = exp2_in_order(x[2 * i + 3]);
        }
        fadd2(l[2 * (i & 1)], l[2 * (i & 1) + 1], x[2 * i], x[2 * i + 1]);
        w[i] = pack_in_order(x[2 * i], x[2 * i + 1]);
    }
    if constexpr (FORM != FORM_PLAIN) {
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const uint32_t u = f32x2_to_bf16x2(x[2 * j] - __uint_as_float(w[j] << 16),
                                               x[2 * j + 1] - __uint_as_float(w[j] & 0xffff0000u));
            if constexpr (FORM == FORM_TWICE) held[j] = u;
            else w[j] = rest ? u : w[j];
        }
    }
    tmem_st16(tP, w);
}

// A tile's scores at tS (this warp's 32 rows, 128 columns) to its weights P
// (64 columns at tS); returns the row's sum.  The scores are read 32 at a time
// (held from the maximum on they would fill the registers); P is handed over
// in two halves, the products of the first running beside the exponentials of
// the second.  One copy per form, and a loop over the halves: the code of a
// tile has to stay in the instruction cache.
template <int FORM>
__device__ __forceinline__ float weights128(uint32_t tS, float sl, float neg, bool rest, uint64_t* some,
                                            uint64_t* more) {
    float ls[4] = {0.f, 0.f, 0.f, 0.f};
    auto hand_over = [&](int half) {
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(half == 0 ? some : more);
    };
    if constexpr (FORM != FORM_TWICE) {
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
            uint32_t x[32], none[16];
            tmem_ld32(tS + c * 32, x);
            tmem_ld_wait();
            weights32<FORM>(x, tS + c * 16, sl, neg, rest, ls, none);
            if (c & 1) hand_over(c >> 1);
        }
    } else {
        // the remainders lie beside P, in columns 64 .. 127: a half's wait
        // until the scores there are in registers
        uint32_t xa[32], xb[32], held[2][16];
        tmem_ld32(tS, xa);
        tmem_ld32(tS + 32, xb);
        tmem_ld_wait();
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
            weights32<FORM>(xa, tS + h * 32, sl, neg, rest, ls, held[0]);
            weights32<FORM>(xb, tS + h * 32 + 16, sl, neg, rest, ls, held[1]);
            if (h == 0) {
                tmem_ld32(tS + 64, xa);
                tmem_ld32(tS + 96, xb);
                tmem_ld_wait();
            }
            tmem_st16(tS + 64 + h * 32, held[0]);
            tmem_st16(tS + 80 + h * 32, held[1]);
            hand_over(h);
        }
    }
    return (ls[0] + ls[1]) + (ls[2] + ls[3]);
}

template <int N>
__device__ __forceinline__ void set_regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void set_regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// S[wg] = Q K^T over D / 16 steps, O[wg] (+)= P V over kTile / 16: one asm
// statement each, the lane elect.sync picks issuing, so that nothing but the
// descriptors' constant steps stands between two products.
__device__ __forceinline__ void issue_qk4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred e, p, q;\n\t.reg .b64 a, b;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "setp.eq.b32 q, 0, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
        "add.s64 a, %1, 2;\n\tadd.s64 b, %2, 2;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, q;\n\t"
        "add.s64 a, %1, 4;\n\tadd.s64 b, %2, 4;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, q;\n\t"
        "add.s64 a, %1, 6;\n\tadd.s64 b, %2, 6;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, q;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
}

__device__ __forceinline__ void issue_pv4(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred e, p, q;\n\t.reg .b64 b;\n\t.reg .b32 a;\n\telect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 q, 0, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
        "add.s32 a, %1, 8;\n\tadd.s64 b, %2, 128;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, q;\n\t"
        "add.s32 a, %1, 16;\n\tadd.s64 b, %2, 256;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, q;\n\t"
        "add.s32 a, %1, 24;\n\tadd.s64 b, %2, 384;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, q;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
}

__device__ __forceinline__ void store_v8(void* to, const uint32_t (&x)[8]) {   // 32 bytes, 32-byte aligned
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(x[0]), "r"(x[1]), "r"(x[2]),
                 "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                 : "memory");
}

// Where a row's output goes: row `at` of out, or (a split block's) row `slot`
// of the workspace.
template <int D>
struct Out {
    bool valid, whole;
    size_t at, slot;
};

// Two at a time: (f0, f1) = (a0, a1) w; (f0, f1) += (a0, a1) w.
__device__ __forceinline__ void scale2(float& f0, float& f1, float a0, float a1, float w) {
    asm("{\n\t.reg .b64 a, w;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 w, {%4, %4};\n\t"
        "mul.rn.f32x2 a, a, w;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "=f"(f0), "=f"(f1)
        : "f"(a0), "f"(a1), "f"(w));
}

__device__ __forceinline__ void add_scaled2(float& f0, float& f1, float a0, float a1, float w) {
    asm("{\n\t.reg .b64 a, f, w;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 f, {%0, %1};\n\tmov.b64 w, {%4, %4};\n\t"
        "fma.rn.f32x2 f, a, w, f;\n\tmov.b64 {%0, %1}, f;\n\t}"
        : "+f"(f0), "+f"(f1)
        : "f"(a0), "f"(a1), "f"(w));
}

// Columns 16 c0 .. 16 c1 - 1 of a warp's 32 rows of O, from tensor memory to
// where they go.  JOINED: w0 O0 + w1 O1 (t1 = 0: no O1); stacked: the lane 16
// on holds the remainders' part.  It runs once a block, so its time is the
// instructions' way into the cache: no copy for each form.
template <int D, bool E4M3, bool JOINED>
__device__ __forceinline__ void put_rows(const AttendParams& p, const Scratch& ws, const Out<D>& to, uint32_t t0,
                                         uint32_t t1, int c0, int c1, float w0, float w1, bool stacked,
                                         const volatile Blk* odd, int m, float m_ref) {
    // out is 16-byte aligned: 32-byte stores where it is more
    const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
    uint32_t o[16], q[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) q[j] = 0;
    tmem_ld16(t0 + c0 * 16, o);
    if (JOINED && t1) tmem_ld16(t1 + c0 * 16, q);
#pragma unroll 1
    for (int c = c0; c < c1; ++c) {
        float f[16];
        tmem_ld_wait();
        // a weight is 0 only where that o is 0 too (no key seen) or absent
#pragma unroll
        for (int j = 0; j < 16; j += 2)
            scale2(f[j], f[j + 1], __uint_as_float(o[j]), __uint_as_float(o[j + 1]), w0);
        if constexpr (JOINED) {
#pragma unroll
            for (int j = 0; j < 16; j += 2)
                add_scaled2(f[j], f[j + 1], __uint_as_float(q[j]), __uint_as_float(q[j + 1]), w1);
        }
        if (c + 1 < c1) {   // the next columns on their way
            tmem_ld16(t0 + (c + 1) * 16, o);
            if (JOINED && t1) tmem_ld16(t1 + (c + 1) * 16, q);
        }
        if (JOINED && stacked) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float y = __shfl_down_sync(0xffffffffu, f[j], 16);
                if (fabsf(f[j]) < INFINITY) f[j] += y;   // a remainder has either sign: not on infinities
            }
        }
        if (__builtin_expect(odd != nullptr && to.valid, 0)) {
            float g[16];
            Blk blk;
            const int4* src = reinterpret_cast<const int4*>(const_cast<const Blk*>(odd));
#pragma unroll
            for (int k = 0; k < 4; ++k) reinterpret_cast<int4*>(&blk)[k] = src[k];
            for (int j = 0; j < 16; ++j) g[j] = 0.f;
            add_nonfinite<D, E4M3>(p, blk, m, m_ref, c * 16, g);
            for (int j = 0; j < 16; ++j) f[j] += g[j];   // scaling would change neither infinities nor NaN
        }
        if (to.whole) {
            uint32_t y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = f32x2_to_bf16x2(f[2 * j], f[2 * j + 1]);
            uint16_t* dst = p.out + to.at * D + c * 16;
            if (to.valid && wide) store_v8(dst, y);
            if (to.valid && !wide) {
                reinterpret_cast<uint4*>(dst)[0] = make_uint4(y[0], y[1], y[2], y[3]);
                reinterpret_cast<uint4*>(dst)[1] = make_uint4(y[4], y[5], y[6], y[7]);
            }
        } else if (to.valid) {
            float* dst = ws.o + to.slot * D + c * 16;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t y[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] = __float_as_uint(f[8 * h + j]);
                store_v8(dst + 8 * h, y);
            }
        }
        __syncwarp();
    }
}

// Reads the handed-out blocks in turn.
template <int BLOCKS>
struct Reader {
    uint32_t n = 0;
    __device__ __forceinline__ int at() const { return n % BLOCKS; }
    __device__ __forceinline__ uint32_t phase() const { return (n / BLOCKS) & 1; }
};

template <int D, bool E4M3, bool SMALL>
__global__ void __launch_bounds__(Cfg<D, E4M3, SMALL>::kThreads, 1)
    attend_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                  const __grid_constant__ CUtensorMap tmQ,
                  const __grid_constant__ AttendParams p, const __grid_constant__ Scratch ws) {
    using C = Cfg<D, E4M3, SMALL>;
    using B = Bars<C::kSlots, C::kRawSlots, C::kRingBlocks>;
    extern __shared__ __align__(1024) uint8_t smem[];
    static_assert(sizeof(B) == C::kNumBars * 8, "barriers");
    B& bar = *reinterpret_cast<B*>(smem + C::kBars);
    Blk* blks = reinterpret_cast<Blk*>(smem + C::kBlks);
    float2* xch = reinterpret_cast<float2*>(smem + C::kXch);
    Start* start = reinterpret_cast<Start*>(smem + C::kXch);               // only until the roles begin
    unsigned long long* wsum = reinterpret_cast<unsigned long long*>(smem + C::kXch + 64);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kMisc);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (warp == 8) {
        if (lane == 0) {
            tma_prefetch_desc(&tmK);
            tma_prefetch_desc(&tmV);
            if (!SMALL) tma_prefetch_desc(&tmQ);
        }
    } else if (warp == 9) {
        tmem_alloc(tmem_slot, kTmemCols);
        tmem_relinquish();
    } else if (warp == 10) {
        for (int k = lane; k < C::kSlots; k += 32) {
            mbar_init(&bar.full[k], E4M3 ? 4 : 1);
            mbar_init(&bar.empty[k], 1);
            if (!E4M3) mbar_init(&bar.dirty[k], 1);
        }
        for (int k = lane; k < C::kRawSlots; k += 32) {
            mbar_init(&bar.raw_full[k], 1);
            mbar_init(&bar.raw_empty[k], 4);
        }
        for (int k = lane; k < C::kRingBlocks; k += 32) {
            mbar_init(&bar.blk_full[k], 1);
            mbar_init(&bar.blk_empty[k], 8 + 3 + (E4M3 ? 8 : 0));   // the warps that read it
        }
        if (lane < 2) {
            mbar_init(&bar.s_full[lane], 1);
            mbar_init(&bar.p_half[lane][0], 4);
            mbar_init(&bar.p_half[lane][1], 4);
            mbar_init(&bar.o_full[lane], 1);
        }
        if (lane == 0) {
            mbar_init(&bar.q_full, 1);
            mbar_init(&bar.q_empty, 1);
            mbar_init(&bar.xch, 8);
            mbar_init(&bar.xdone, 8);
            mbar_init(&bar.drain, 1);
        }
        fence_mbar_init();
    }
    pdl_wait();
    pdl_trigger();
    // a few small requests: the walking warp finds the start by itself, later
    // (one token over 500 keys 12.5 us against 14.0 with all warps, 32 trees of
    // 65 slots 134 against 135); beyond 32 it would need several rounds
    const bool by_all = p.R > 32 || p.max_window * p.group > 4 * p.sub;
    if (by_all) plan<C::kThreads>(p, reinterpret_cast<unsigned long long*>(smem + C::kRing), start, wsum);
    Start st = *start;   // read before the roles use its place
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    Reader<C::kRingBlocks> rd;
    // waits for the next block; its entry stays valid until release()
    auto take = [&](bool& ok) -> const volatile Blk* {
        ok = wait_or_fail(p, &bar.blk_full[rd.at()], rd.phase());
        if (!ok) return nullptr;
        const volatile Blk* b = blks + rd.at();
        return b->t1 > 0 ? b : nullptr;
    };
    auto release = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.blk_empty[rd.at()]);
        ++rd.n;
    };
    auto copy = [](const volatile Blk* b) {
        Blk r;
        const int4* src = reinterpret_cast<const int4*>(const_cast<const Blk*>(b));
        int4* dst = reinterpret_cast<int4*>(&r);
#pragma unroll
        for (int k = 0; k < 4; ++k) dst[k] = src[k];
        return r;
    };

    if (warp < 8) {
        // ------------------------------------------------------------------
        // softmax warpgroups
        // ------------------------------------------------------------------
        set_regs_up<C::kRegsSoft>();
        const int wg = warp >> 2, row = tid & 127;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lanes + wg * 128;
        const uint32_t tO0 = tmem + lanes + 256, tO1 = tO0 + 128;
        const uint32_t tO = wg ? tO1 : tO0;
        const float sl = p.scale * kLog2e;
        uint32_t n_s = 0, n_o0 = 0, n_o1 = 0, n_x = 0;   // phases of s_full, o_full, xch and xdone
        bool ok, x_open = false;
        Share share = {};
        share.head = 3;
        for (;;) {
            const volatile Blk* vb = take(ok);
            if (!vb) break;
            const int flags = vb->flags, M = vb->M, m0 = vb->m0, t0 = vb->t0;
            const bool pair = !SMALL && (flags & BLK_PAIR);
            const bool stacked = flags & BLK_STACKED, twice = !SMALL && (flags & BLK_TWICE);
            const int n_tiles = vb->t1 - t0;
            const bool rest = stacked && (lane & 16);             // this lane holds the weights' remainders
            const int r = stacked ? (row >> 5) * 16 + (row & 15) : pair ? wg * p.sub + row : row;   // row of the block
            const int lim = pair ? min(M, (wg + 1) * p.sub) : M;  // its warpgroup's rows end here
            const bool busy = (stacked ? r & ~15 : r - lane) < lim;   // the warp has rows
            float m_ref = -INFINITY, l = 0.f;
            {
                const int ctx = vb->ctx, n_rows = vb->n, ns = vb->ns, lo = vb->lo;
                const int first_m = m0 + (pair ? wg * p.sub : 0);
                const int p0 = pair ? first_m / p.group : vb->p0;
                const int p1 = pair ? (min(first_m + p.sub, m0 + M) - 1) / p.group : vb->p1;
                const RowView view = row_view(p, vb->i, ctx, n_rows, min((m0 + r) / p.group, n_rows - 1));
                const int mine = pair ? n_tiles : (n_tiles + 1 - wg) >> 1;
                for (int it = 0; it < mine; ++it) {
                    const int t = t0 + (pair ? it : 2 * it + wg);
                    const int key0 = (t < ns ? t : lo + t - ns) * kTile;
                    const bool mixed = tile_mixed(p, ctx, p0, p1, key0);
                    ok = wait_or_fail(p, &bar.s_full[wg], n_s & 1);
                    ++n_s;
                    if (!ok) break;
                    tc_fence_after();
                    if (busy) {
                        float top;
                        if (__builtin_expect(mixed, 0)) {
                            // few tiles: their scores are masked where they stand
                            top = -INFINITY;
#pragma unroll 1
                            for (int c = 0; c < 4; ++c) {
                                uint32_t y[32];
                                tmem_ld32(tS + c * 32, y);
                                const uint32_t see = seen32(view, key0 + 32 * c);
                                tmem_ld_wait();
                                if (!__all_sync(0xffffffffu, see == 0xffffffffu)) {
#pragma unroll
                                    for (int j = 0; j < 32; ++j)
                                        if (!((see >> j) & 1u)) y[j] = 0xff800000u;
                                    tmem_st32(tS + c * 32, y);
                                }
                                float z = -INFINITY;
#pragma unroll
                                for (int j = 0; j < 32; j += 4) {
                                    top = max3(top, __uint_as_float(y[j]), __uint_as_float(y[j + 1]));
                                    z = max3(z, __uint_as_float(y[j + 2]), __uint_as_float(y[j + 3]));
                                }
                                top = fmaxf(top, z);
                            }
                            top *= sl;
                            tmem_st_wait();
                        } else {
                            top = tile_max<2>(tS) * sl;
                        }
                        // only lanes that hold a row of the block have a say: what the others'
                        // scores come from is left in shared memory by whatever ran before
                        if (__builtin_expect(__any_sync(0xffffffffu, r < lim && top > m_ref + kLazy), 0)) {
                            const float to = fminf(fmaxf(m_ref, top), kMaxRef);
                            const float corr = to == -INFINITY ? 1.f : fast_exp2(m_ref - to);
                            m_ref = to;
                            l *= corr;
                            if (it > 0) {
                                // the tile before has been added: S of this one was
                                // issued after that product and has completed
#pragma unroll 1
                                for (int c = 0; c < D / 32; ++c) {
                                    uint32_t o[32];
                                    tmem_ld32(tO + c * 32, o);
                                    tmem_ld_wait();
#pragma unroll
                                    for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * corr);
                                    tmem_st32(tO + c * 32, o);
                                }
                            }
                        }
                    }
                    if (__builtin_expect(x_open, 0)) {
                        // the other warpgroup has read this one's O of the block before
                        ok = wait_or_fail(p, &bar.xdone, (n_x - 1) & 1);
                        x_open = false;
                        if (!ok) break;
                    }
                    const float neg = m_ref == -INFINITY ? 0.f : -m_ref;
                    if (busy) {
                        uint64_t* some = &bar.p_half[wg][0];
                        uint64_t* more = &bar.p_half[wg][1];
                        if (stacked) l += weights128<FORM_STACKED>(tS, sl, neg, rest, some, more);
                        else if (twice) l += weights128<FORM_TWICE>(tS, sl, neg, rest, some, more);
                        else l += weights128<FORM_PLAIN>(tS, sl, neg, rest, some, more);
                    } else {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(&bar.p_half[wg][0]);
                            mbar_arrive(&bar.p_half[wg][1]);
                        }
                    }
                }
            }
            if (!ok) break;
            // ---- the block's end -------------------------------------------
            const int all = vb->tiles;
            const bool whole = t0 == 0 && n_tiles == all;
            const size_t slot = 2 * static_cast<size_t>(blockIdx.x) + (t0 > 0 ? 0 : 1);
            if (tid == 0) {
                if (rd.n == 0) share.head = t0 == 0 ? 0 : t0 + n_tiles == all ? 1 : 2;
                if (t0 == 0 && !whole) {
                    share.rows = M;
                    share.row0 = vb->row0;
                    share.m0 = m0;
                    share.hk = vb->hk;
                }
            }
            float a0 = 1.f, a1 = 0.f;      // weights of the first and the second warpgroup's o
            const bool joined = !pair;
            if (joined) {
                if (x_open) {              // only a block in which this warpgroup had no tile leaves it open
                    ok = wait_or_fail(p, &bar.xdone, (n_x - 1) & 1);
                    x_open = false;
                    if (!ok) break;
                }
                if (!SMALL || (!rest && r < kStackRows))
                    xch[wg * C::kXchRows + (SMALL ? r : row)] = make_float2(m_ref, l);
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.xch);
                ok = wait_or_fail(p, &bar.xch, n_x & 1);
                if (!ok) break;
                const float2 other = xch[(wg ^ 1) * C::kXchRows + (SMALL ? min(r, kStackRows - 1) : row)];
                const float mm = fmaxf(m_ref, other.x);
                const float ref = mm == -INFINITY ? 0.f : mm;
                const float b0 = m_ref == -INFINITY ? 0.f : fast_exp2(m_ref - ref);
                const float b1 = other.x == -INFINITY ? 0.f : fast_exp2(other.x - ref);
                l = l * b0 + other.y * b1;
                m_ref = mm;
                a0 = wg ? b1 : b0;
                a1 = wg ? b0 : b1;
                ok = wait_or_fail(p, &bar.o_full[0], n_o0 & 1);
                if (ok && n_tiles > 1) ok = wait_or_fail(p, &bar.o_full[1], n_o1 & 1);
                ++n_o0;
                n_o1 += n_tiles > 1;
            } else {
                ok = wait_or_fail(p, &bar.o_full[wg], (wg ? n_o1 : n_o0) & 1);
                ++n_o0;
                ++n_o1;
            }
            if (!ok) break;
            tc_fence_after();
            if (busy) {
                const int m = m0 + r, wp = m / p.group;
                Out<D> to;
                to.valid = r < lim && !rest;
                to.whole = whole;
                to.at = (static_cast<size_t>(vb->row0) + wp) * p.H + vb->hk * p.group + (m - wp * p.group);
                to.slot = slot * ws.cap + r;
                if (whole) {
                    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);   // NaN stays NaN
                    a0 *= inv;
                    a1 *= inv;
                }
                const volatile Blk* odd = vb->nonfinite ? vb : nullptr;
                const bool two = joined && n_tiles > 1;   // else the second warpgroup's o was never written
                if (pair) put_rows<D, E4M3, false>(p, ws, to, tO, 0, 0, D / 16, a0, 0.f, false, odd, m, m_ref);
                else
                    put_rows<D, E4M3, true>(p, ws, to, tO0, two ? tO1 : 0, wg * (D / 32), (wg + 1) * (D / 32), a0, a1,
                                            stacked, odd, m, m_ref);
                if (to.valid && (!joined || wg == 0)) {
                    if (!whole) ws.ml[to.slot] = make_float2(m_ref, l);
                    else if (p.lse) p.lse[to.at] = l == 0.f ? -INFINITY : m_ref * kLn2 + logf(l);
                }
            }
            tc_fence_before();   // O has been read before the next block's products are let go
            if (joined) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.xdone);
                ++n_x;
                x_open = true;
            }
            release();
        }
        if (tid == 0) ws.share[blockIdx.x] = share;
    } else if (warp < 12) {
        set_regs_down<C::kRegsRest>();
        bool ok = true;
        if (warp == 11) {
            // ----------------------------------------------------------------
            // producer: K and V tiles in turn, a lane per page.  Not the warp that
            // shares its scheduler with the first warps of the softmax, the only
            // busy ones of small windows (two contexts of 150001 to 199999 101.6
            // us against 104.3)
            // ----------------------------------------------------------------
            const int pages = kTile >> p.c.page_shift, page = 1 << p.c.page_shift;
            constexpr int kN = E4M3 ? C::kRawSlots : C::kSlots;
            constexpr int kRow = E4M3 ? D : 128;          // bytes of a shared-memory row
            uint64_t* full = E4M3 ? bar.raw_full : bar.full;
            uint64_t* empty = E4M3 ? bar.raw_empty : bar.empty;
            uint32_t n = 0, dirty = 0, odd_full = 0, odd_dirty = 0;   // per slot: the barrier armed last, phases mod 2
            int s = 0;
            uint32_t turn = 0;
            for (;;) {
                const volatile Blk* vb = take(ok);
                if (!vb) break;
                const Blk b = copy(vb);
                release();
                const int len = b.ctx + b.n;
                for (int t = b.t0; t < b.t1 && ok; ++t) {
                    const int key0 = tile_key(b, t);
                    const bool cleaned = !E4M3 && tile_cleaned(p, b, key0);
                    const int live = min(pages, (len - key0 + page - 1) >> p.c.page_shift);
                    int pg = 0;
                    if (lane < live) {
                        pg = page_of(p.c, b.i, key0 + lane * page);
                        if (pg < 0) {
                            set_status(p.dev_status, SDM_DEV_BAD_PAGE);
                            pg = 0;
                        }
                    }
                    const int y = (pg * p.c.heads + b.hk) << p.c.page_shift;
                    const uint32_t bytes = static_cast<uint32_t>(live) * page * (E4M3 ? D + 1 : 2 * D);
                    for (int v = 0; v < 2; ++v) {
                        if (turn > 0) ok = wait_or_fail(p, &empty[s], (turn - 1) & 1);
                        if (!ok) break;
                        const bool to_dirty = cleaned && v == 1;
                        uint64_t* arrive = to_dirty ? &bar.dirty[s] : &full[s];
                        const uint32_t bit = 1u << s;
                        dirty = to_dirty ? dirty | bit : dirty & ~bit;
                        if (to_dirty) odd_dirty ^= bit;
                        odd_full ^= bit;
                        if (lane == 0) mbar_arrive_expect_tx(arrive, bytes);
                        __syncwarp();
                        if (lane < live) {
                            if constexpr (E4M3) {
                                tma_load_2d(smem + C::kRaw + s * C::kRawBytes + lane * page * kRow, v ? &tmV : &tmK,
                                            arrive, 0, y);
                                bulk_load(smem + C::kExps + s * kTile + lane * page, (v ? p.c.v_exp : p.c.k_exp) + y,
                                          page, arrive);
                            } else {
#pragma unroll
                                for (int h = 0; h < D / 64; ++h)
                                    tma_load_2d(smem + C::kRing + s * C::kTileBytes + h * (kTile * 128) +
                                                    lane * page * kRow,
                                                v ? &tmV : &tmK, arrive, h * 64, y);
                            }
                        }
                        __syncwarp();
                        ++n;
                        if (++s == kN) {
                            s = 0;
                            ++turn;
                        }
                    }
                }
                if (!ok) break;
            }
            if (!ok) {
                // copies in flight land before the CTA may exit
                for (uint32_t k = 0; k < kN && k < n; ++k) {
                    if ((dirty >> k) & 1u) mbar_wait(&bar.dirty[k], ((odd_dirty >> k) & 1u) ^ 1u);
                    else mbar_wait(&full[k], ((odd_full >> k) & 1u) ^ 1u);
                }
            }
        } else if (warp == 9) {
            // ----------------------------------------------------------------
            // products
            // ----------------------------------------------------------------
            constexpr uint32_t kIdQK = idesc_bf16_f32(kTile, kTile, false);
            constexpr uint32_t kIdPV = idesc_bf16_f32(kTile, D, true);
            const uint64_t q_desc = smem_desc_sw128(smem_u32(smem), 16, 1024);
            const uint64_t k_desc = smem_desc_sw128(smem_u32(smem + C::kRing), 16, 1024);
            const uint64_t v_desc = smem_desc_sw128(smem_u32(smem + C::kRing), kTile * 128, 1024);
            uint32_t n_q = 0, p_phase = 0, full_phase = 0;
            int sk = 0, sv = 1;    // slots of the next K tile and the next V tile to be multiplied
            auto wait_full = [&](int s) {
                const bool r = wait_or_fail(p, &bar.full[s], (full_phase >> s) & 1);
                full_phase ^= 1u << s;
                return r;
            };
            auto next = [&](int s) { return s + 2 >= C::kSlots ? s + 2 - C::kSlots : s + 2; };
            // S = Q K^T
            auto qk = [&](int wg, int q) {
                uint64_t a = q_desc + static_cast<uint64_t>(q * (C::kQBytes >> 4));
                uint64_t b = k_desc + static_cast<uint64_t>(sk * (C::kTileBytes >> 4));
                tc_fence_after();
#pragma unroll 1
                for (int d = 0; d < D / 64; ++d, a += (kTile * 128) >> 4, b += (kTile * 128) >> 4)
                    issue_qk4(tmem + wg * 128, a, b, kIdQK, d > 0);
                mma_commit_warp(&bar.s_full[wg]);
            };
            // waits for P and issues O (+)= P V, half a tile at a time; with
            // the remainders' P, 64 columns on, too
            auto pv = [&](int wg, bool add, bool twice) {
                uint64_t b = v_desc + static_cast<uint64_t>(sv * (C::kTileBytes >> 4));
                uint32_t a = tmem + wg * 128;
#pragma unroll 1
                for (int h = 0; h < 2; ++h, a += 32, b += 512) {
                    if (!wait_or_fail(p, &bar.p_half[wg][h], (p_phase >> wg) & 1)) return false;
                    tc_fence_after();
#pragma unroll 1
                    for (int r = 0; r <= static_cast<int>(twice); ++r) {
                        issue_pv4(tmem + 256 + wg * 128, a + r * 64, b, kIdPV, add);
                        add = true;
                    }
                }
                p_phase ^= 1u << wg;
                return true;
            };
            for (;;) {
                const volatile Blk* vb = take(ok);
                if (!vb) break;
                const int n = vb->t1 - vb->t0, flags = vb->flags;
                release();
                const bool twice = !SMALL && (flags & BLK_TWICE);
                ok = wait_or_fail(p, &bar.q_full, n_q & 1);
                ++n_q;
                if (!ok) break;
                // Per tile and warpgroup: P V of its tile before, then the scores
                // that take its place.  A pair's warpgroups have every tile,
                // else they take turns.
                const bool pair = !SMALL && (flags & BLK_PAIR);
                const int lag = pair ? 1 : 2;
#pragma unroll 1
                for (int t = 0; t < n + lag; ++t) {
                    if (t >= lag) ok = wait_full(sv);
                    if (!ok) break;
#pragma unroll 1
                    for (int k = 0; k < (pair ? 2 : 1); ++k) {
                        const int wg = pair ? k : t & 1;
                        if (t >= lag) {
                            ok = pv(wg, t >= 2 * lag, twice);
                            if (!ok) break;
                            if (t >= n) mma_commit_warp(&bar.o_full[wg]);
                        }
                        if (t < n) {
                            if (k == 0) ok = wait_full(sk);
                            if (!ok) break;
                            qk(wg, pair ? k : 0);
                        }
                    }
                    if (!ok) break;
                    if (t < n) {
                        mma_commit_warp(&bar.empty[sk]);
                        sk = next(sk);
                    }
                    if (t >= lag) {
                        mma_commit_warp(&bar.empty[sv]);
                        sv = next(sv);
                    }
                    if (t == n - 1) mma_commit_warp(&bar.q_empty);
                }
                if (!ok) break;
            }
            if (!ok) {   // this warp's own tensor-core work ends before tensor memory is freed
                mma_commit_warp(&bar.drain);
                mbar_wait(&bar.drain, 0);
            }
        } else if (warp == 10) {
            // ----------------------------------------------------------------
            // Q rows of each block: a sub-tile is one box of whole tokens, the rows
            // of a stacked block go to two places, a lane each; bf16: then the
            // values of the tiles to be cleared, a key's row per lane
            // ----------------------------------------------------------------
            uint32_t n_q = 0, dirty_phase = 0;
            int sv = 1;            // slot of the next V tile
            for (;;) {
                const volatile Blk* vb = take(ok);
                if (!vb) break;
                const int row0 = vb->row0, m0 = vb->m0, M = vb->M, hk = vb->hk;
                const bool stacked = vb->flags & BLK_STACKED;
                if (n_q > 0) ok = wait_or_fail(p, &bar.q_empty, (n_q - 1) & 1);
                ++n_q;
                if (!ok) break;
                const bool boxes = !SMALL && !stacked;
                if (boxes) {
                    if (lane == 0) {
                        const int subs = (vb->flags & BLK_PAIR) ? 2 : 1;
                        mbar_arrive_expect_tx(&bar.q_full, subs * p.sub * D * 2);
                        for (int k = 0; k < subs; ++k)
#pragma unroll
                            for (int h = 0; h < D / 64; ++h)
                                tma_load_3d(smem + k * C::kQBytes + h * (kTile * 128), &tmQ, &bar.q_full, h * 64,
                                            hk * p.group, row0 + (m0 + k * p.sub) / p.group);
                    }
                    __syncwarp();
                }
                for (int r = lane; !boxes && r < M; r += 32) {
                    const int m = m0 + r, wp = m / p.group;
                    const uint16_t* src = p.q + (row0 + wp) * p.q_stride +
                                          static_cast<size_t>(hk * p.group + (m - wp * p.group)) * D;
                    const int to = stacked ? (r >> 4) * 32 + (r & 15) : r;   // 16 rows on keeps r mod 8 and the swizzle
                    const uint32_t dst = to * 128 + ((to & 7) << 4);
#pragma unroll
                    for (int c = 0; c < D / 8; ++c) {
                        uint8_t* d = smem + (c >> 3) * (kTile * 128) + (dst ^ ((c & 7) << 4));
                        cp_async_16(d, src + c * 8, 16u);
                        if (stacked) cp_async_16(d + 16 * 128, src + c * 8, 16u);
                    }
                }
                if (!boxes) {
                    cp_async_wait_all();
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.q_full);
                }
                if constexpr (!E4M3) {
                    const Blk b = copy(vb);
                    const int len = b.ctx + b.n;
                    for (int t = b.t0; t < b.t1; ++t) {
                        const int key0 = tile_key(b, t), s = sv;
                        sv = sv + 2 >= C::kSlots ? sv + 2 - C::kSlots : sv + 2;
                        if (!tile_cleaned(p, b, key0)) continue;
                        ok = wait_or_fail(p, &bar.dirty[s], (dirty_phase >> s) & 1);
                        dirty_phase ^= 1u << s;
                        if (!ok) break;
                        bool found = false;
#pragma unroll 1
                        for (int row = lane; row < kTile * (D / 64); row += 32) {
                            uint4* v = reinterpret_cast<uint4*>(smem + C::kRing + s * C::kTileBytes + row * 128);
                            uint4 x[8];
                            // pieces in an order that keeps the lanes of a quarter-warp on different banks
#pragma unroll
                            for (int c = 0; c < 8; ++c) x[c] = v[c ^ (row & 7)];
                            uint32_t any = 0;
#pragma unroll
                            for (int c = 0; c < 8; ++c)
                                any |= nonfinite2(x[c].x) | nonfinite2(x[c].y) | nonfinite2(x[c].z) |
                                       nonfinite2(x[c].w);
                            if (__builtin_expect(any != 0, 0)) {
                                uint32_t* u = reinterpret_cast<uint32_t*>(v);
#pragma unroll 1
                                for (int j = 0; j < 32; ++j) {
                                    const uint32_t bad = nonfinite2(u[j]);
                                    if (bad & 0x8000u) u[j] &= 0xffff0000u;
                                    if (bad & 0x80000000u) u[j] &= 0xffffu;
                                }
                                found |= key0 + (row & (kTile - 1)) < len;
                            }
                        }
                        if (found) blks[rd.at()].nonfinite = 1;
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bar.full[s]);
                    }
                    if (!ok) break;
                }
                release();
            }
            if (!ok && n_q > 0) mbar_wait(&bar.q_full, (n_q - 1) & 1);   // a copy in flight lands first
        } else {
            // ----------------------------------------------------------------
            // the share's blocks, in turn, for the other warps
            // ----------------------------------------------------------------
            if (!by_all) plan_few(p, st);
            Walk k;
            k.init(st);
            bool more = st.u0 < st.u1;
            for (uint32_t n = 0;; ++n) {
                more = more && k.next(p);
                const int e = n % C::kRingBlocks;
                if (n >= C::kRingBlocks && !wait_or_fail(p, &bar.blk_empty[e], ((n / C::kRingBlocks) - 1) & 1)) break;
                if (lane == 0) {
                    Blk b = {};
                    if (more) {
                        b.i = k.i;
                        b.hk = k.hk;
                        b.row0 = k.w.row0;
                        b.n = k.w.n;
                        b.ctx = k.w.ctx;
                        b.m0 = k.g.m0;
                        b.M = k.g.M;
                        b.p0 = k.g.p0;
                        b.p1 = k.g.p1;
                        b.ns = k.g.ns;
                        b.lo = k.g.lo;
                        b.tiles = k.g.n;
                        b.t0 = k.t0;
                        b.t1 = k.t1;
                        b.flags = (k.g.pair ? BLK_PAIR : 0) | (k.g.stacked ? BLK_STACKED : 0) |
                                  (k.g.twice ? BLK_TWICE : 0);
                    }
                    blks[e] = b;
                    mbar_arrive(&bar.blk_full[e]);
                }
                __syncwarp();
                if (!more) break;
            }
        }
    } else {
        // --------------------------------------------------------------------
        // e4m3 codes -> bf16 values, a key's row per thread; one warpgroup takes
        // the K tiles, the other the V tiles.  A tile takes a warpgroup about
        // 1900 clocks, its instructions' rate beside the other's (two warpgroups
        // a tile: slower, 106 -> 118 us for two contexts of 150001 to 199999);
        // two pieces a step is what the instruction cache holds (one: 110 us,
        // four: 104 us there, but 256 windows 155 -> 188 us)
        // --------------------------------------------------------------------
        if constexpr (E4M3) {
            set_regs_down<C::kRegsRest>();
            bool ok = true;
            const int row = tid & 127, v = (tid >> 7) - 3;
            int s = v, rs = v;
            uint32_t turn = 0, raw_turn = 0;
            for (;;) {
                const volatile Blk* vb = take(ok);
                if (!vb) break;
                const Blk b = copy(vb);
                const int len = b.ctx + b.n;
                for (int t = b.t0; t < b.t1; ++t) {
                    const int key0 = tile_key(b, t);
                    const bool clear = v == 1 && tile_cleaned(p, b, key0);
                    {
                        ok = wait_or_fail(p, &bar.raw_full[rs], raw_turn & 1);
                        if (ok && turn > 0) ok = wait_or_fail(p, &bar.empty[s], (turn - 1) & 1);
                        if (!ok) break;
                        // the TMA swizzle: 16-byte piece c of row r sits at c ^ (r mod 8), rows of 64
                        // bytes at c ^ (r / 2 mod 4); a bf16 row's pieces 2 c and 2 c + 1 likewise
                        const int src = C::kRaw + rs * C::kRawBytes + row * D +
                                        (D == 128 ? (row & 7) : ((row >> 1) & 3)) * 16;
                        const int dst = C::kRing + s * C::kTileBytes + row * 128 + (row & 7) * 16;
                        const uint32_t e = smem[C::kExps + rs * kTile + row];
                        // 2^(e - 127) as bf16, twice
                        const uint32_t sc = scale_byte(e) << 7;
                        const uint32_t scale2 = sc | (sc << 16);
                        uint4 x = *reinterpret_cast<const uint4*>(smem + src);
#pragma unroll 2
                        for (int c = 0; c < D; c += 16) {
                            const uint32_t u[4] = {x.x, x.y, x.z, x.w};
                            // the next piece's load runs under this one's arithmetic
                            x = *reinterpret_cast<const uint4*>(smem + (src ^ ((c + 16) & (D - 1))));
                            uint32_t o[8];
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const float2 f = f16x2_to_f32x2(
                                    e4m3x2_to_f16x2(static_cast<uint16_t>(u[j >> 1] >> (16 * (j & 1)))));
                                uint32_t y = f32x2_to_bf16x2(f.x, f.y);
                                asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(y) : "r"(scale2));
                                o[j] = y;
                            }
                            const int to = (dst + (c >> 6) * (kTile * 128)) ^ ((2 * c) & 127);
                            *reinterpret_cast<uint4*>(smem + to) = make_uint4(o[0], o[1], o[2], o[3]);
                            *reinterpret_cast<uint4*>(smem + (to ^ 16)) = make_uint4(o[4], o[5], o[6], o[7]);
                            if (clear) {
                                uint32_t bad = 0;   // bits 15 and 31: an exponent field of ones
#pragma unroll
                                for (int j = 0; j < 8; ++j) bad |= (o[j] & 0x7fff7fffu) + 0x00800080u;
                                if (__builtin_expect((bad & 0x80008000u) != 0, 0)) {
                                    if (key0 + row < len) blks[rd.at()].nonfinite = 1;
#pragma unroll 1
                                    for (int j = 0; j < 8; ++j) {
                                        uint32_t* y = reinterpret_cast<uint32_t*>(smem + (to ^ (j * 4)));
                                        bad = nonfinite2(*y);
                                        if (bad & 0x8000u) *y &= 0xffff0000u;
                                        if (bad & 0x80000000u) *y &= 0xffffu;
                                    }
                                }
                            }
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(&bar.raw_empty[rs]);
                            mbar_arrive(&bar.full[s]);
                        }
                        s += 2;
                        if (s >= C::kSlots) {
                            s -= C::kSlots;
                            ++turn;
                        }
                        rs += 2;
                        if (rs >= C::kRawSlots) {
                            rs -= C::kRawSlots;
                            ++raw_turn;
                        }
                    }
                }
                if (!ok) break;
                release();
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// Joins the segments of split blocks, in key order: the CTA whose share
// starts a block and the next ones that continue it.  kRows rows a warp, the
// loads of kSegs segments together: the kernel is a chain of a few L2 round
// trips (bytes: at most 2 x 256 rows x 4 D per CTA, written and read once).
// Small windows are long contexts over many CTAs, so 8 segments of a row: two
// contexts of 150001 to 199999 (38 segments) take 102 us against 109 with a
// segment at a time (4: 104; 16: 101, but 64 windows 108 against 106).  Larger
// ones have two or three segments and many rows, so 2 rows: five e4m3 windows
// 66.4 us (a row at a time: 67.5).
template <int D, int kRows, int kSegs>
__global__ void __launch_bounds__(256) attend_merge_kernel(const AttendParams p, const Scratch ws, int grid) {
    constexpr int kV = D / 32;
    pdl_wait();
    pdl_trigger();
    const int c = blockIdx.x, lane = threadIdx.x & 31;
    const Share s = ws.share[c];
    // slots of the block: 2c + 1, then slot 0 of the CTAs after c up to the one that finishes it
    int end = c + 1;
    unsigned none = 0;     // of the first 32 of them: without work
    for (bool first = true;; first = false) {
        const int at = end + lane;
        const int head = at < grid ? ws.share[at].head : 1;
        if (s.rows == 0) return;
        if (first) none = __ballot_sync(0xffffffffu, head == 3);
        const unsigned stop = __ballot_sync(0xffffffffu, head == 1 || head == 0);
        if (stop) {
            end += __ffs(stop);
            break;
        }
        end += 32;
    }
    end = min(end, grid);
    const int r0 = (blockIdx.y * 8 + (threadIdx.x >> 5)) * kRows;
    if (r0 >= s.rows) return;
    float m[kRows], l[kRows], o[kRows][kV];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int j = 0; j < kV; ++j) o[r][j] = 0.f;
    }
    for (int k0 = c; k0 < end; k0 += kSegs) {
        float2 ml[kSegs][kRows];
        float x[kSegs][kRows][kV];
#pragma unroll
        for (int g = 0; g < kSegs; ++g) {
            const int k = k0 + g;
            const bool idle = k > c && k < end && (k - c <= 32 ? (none >> (k - c - 1)) & 1u : ws.share[k].head == 3);
            const bool work = k < end && !idle;
            const size_t slot = (k == c ? 2 * static_cast<size_t>(c) + 1 : 2 * static_cast<size_t>(k)) * ws.cap + r0;
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                ml[g][r] = make_float2(-INFINITY, 0.f);
                if (!work || r0 + r >= s.rows) continue;
                ml[g][r] = ws.ml[slot + r];
                const float* src = ws.o + (slot + r) * D + lane * kV;
                if constexpr (kV == 4) {
                    const float4 t = *reinterpret_cast<const float4*>(src);
                    x[g][r][0] = t.x, x[g][r][1] = t.y, x[g][r][2] = t.z, x[g][r][3] = t.w;
                } else {
                    const float2 t = *reinterpret_cast<const float2*>(src);
                    x[g][r][0] = t.x, x[g][r][1] = t.y;
                }
            }
        }
#pragma unroll
        for (int g = 0; g < kSegs; ++g) {
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                if (ml[g][r].x == -INFINITY && ml[g][r].y == 0.f) continue;
                const float to = fmaxf(m[r], ml[g][r].x);
                const float a = m[r] == -INFINITY ? 0.f : fast_exp2(m[r] - to), b = fast_exp2(ml[g][r].x - to);
                m[r] = to;
                l[r] = l[r] * a + ml[g][r].y * b;
#pragma unroll
                for (int j = 0; j < kV; ++j) o[r][j] = o[r][j] * a + x[g][r][j] * b;
            }
        }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        if (r0 + r >= s.rows) break;
        const int mm = s.m0 + r0 + r;
        const size_t at = (static_cast<size_t>(s.row0) + mm / p.group) * p.H + s.hk * p.group + mm % p.group;
        const float inv = l[r] > 0.f ? 1.f / l[r] : (l[r] == 0.f ? 0.f : l[r]);
        uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + at * D + lane * kV);
        if constexpr (kV == 4)
            *reinterpret_cast<uint2*>(dst) = make_uint2(f32x2_to_bf16x2(o[r][0] * inv, o[r][1] * inv),
                                                        f32x2_to_bf16x2(o[r][2] * inv, o[r][3] * inv));
        else
            *dst = f32x2_to_bf16x2(o[r][0] * inv, o[r][1] * inv);
        if (lane == 0 && p.lse) p.lse[at] = l[r] == 0.f ? -INFINITY : m[r] * kLn2 + logf(l[r]);
    }
}

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

int slot_rows(int max_window, int group) {
    const long long m = static_cast<long long>(max_window) * group;
    return m >= 2 * kTile ? 2 * kTile : static_cast<int>((m + 7) & ~7ll);
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    if (!fn) {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    }
    return fn;
}

// q as (dim, head, row): a box is 64 dims of the heads of one kv head and as
// many tokens as a sub-tile holds, which land as the sub-tile's rows.
bool encode_q(CUtensorMap* map, const AttendParams& p) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(p.c.D), static_cast<cuuint64_t>(p.H),
                          static_cast<cuuint64_t>(p.rows)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(p.c.D) * 2, static_cast<cuuint64_t>(p.q_stride) * 2};
    cuuint32_t box[3] = {64u, static_cast<cuuint32_t>(p.group), static_cast<cuuint32_t>(p.sub / p.group)};
    cuuint32_t el[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(p.q), dims, strides, box, el,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode(CUtensorMap* map, const CacheView& c, void* pool) {
    auto fn = encode_fn();
    if (!fn) return false;
    // rows = (page, head, slot); a box is one page of one head, 128 bytes (e4m3 with 64-wide heads: 64) across
    const int es = c.e4m3 ? 1 : 2;
    const int cols = c.e4m3 ? c.D : 64;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(c.D),
                          static_cast<cuuint64_t>(c.n_pages) * c.heads << c.page_shift};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(c.D) * es};
    cuuint32_t box[2] = {static_cast<cuuint32_t>(cols), 1u << c.page_shift};
    cuuint32_t el[2] = {1, 1};
    return fn(map, c.e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, pool, dims, strides,
              box, el, CU_TENSOR_MAP_INTERLEAVE_NONE,
              cols * es == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool E4M3, bool SMALL>
cudaError_t launch_one(const AttendParams& p, void* work, cudaStream_t s) {
    using C = Cfg<D, E4M3, SMALL>;
    static bool configured = false;
    if (!configured) {
        const cudaError_t e = cudaFuncSetAttribute(attend_kernel<D, E4M3, SMALL>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, C::kTotal);
        if (e != cudaSuccess) return e;
        configured = true;
    }
    CUtensorMap tmK, tmV;
    if (!encode(&tmK, p.c, p.c.k) || !encode(&tmV, p.c, p.c.v)) return cudaErrorInvalidValue;
    CUtensorMap tmQ = tmK;
    if (!SMALL && !encode_q(&tmQ, p)) return cudaErrorInvalidValue;
    const int grid = num_sms();
    Scratch ws;
    uint8_t* at = static_cast<uint8_t*>(work);
    ws.cap = slot_rows(p.max_window, p.group);
    ws.share = reinterpret_cast<Share*>(at);
    at += align256(sizeof(Share) * grid);
    ws.ml = reinterpret_cast<float2*>(at);
    at += align256(2 * static_cast<size_t>(grid) * ws.cap * sizeof(float2));
    ws.o = reinterpret_cast<float*>(at);
    cudaError_t e =
        launch_pdl(attend_kernel<D, E4M3, SMALL>, dim3(grid), dim3(C::kThreads), C::kTotal, s, tmK, tmV, tmQ,
                   p, ws);
    if (e != cudaSuccess) return e;
    constexpr int kRows = SMALL ? 1 : 2, kSegs = SMALL ? 8 : 1;
    return launch_pdl(attend_merge_kernel<D, kRows, kSegs>, dim3(grid, (ws.cap + 8 * kRows - 1) / (8 * kRows)),
                      dim3(256), 0, s, p, ws, grid);
}

}  // namespace

size_t attend_workspace(int max_window, int H, int D, int kv_heads) {
    if (max_window <= 0 || H <= 0 || D <= 0 || kv_heads <= 0) return 0;
    const size_t grid = num_sms(), cap = slot_rows(max_window, (H + kv_heads - 1) / kv_heads);
    return align256(sizeof(Share) * grid) + align256(2 * grid * cap * sizeof(float2)) + 2 * grid * cap * D * 4;
}

// SMALL: every block has at most kStackRows rows, so one sub-tile of Q and the
// stream form do, and the shared memory of the other goes to the ring.
template <int D, bool E4M3>
static cudaError_t launch_form(const AttendParams& p, void* ws, cudaStream_t s) {
    // Costs of the shares' units, about 0.1 us each, fitted to the times of the
    // CTAs' shares: a block besides its tiles (Q, the first product, the last
    // O; 3.5 to 8 us), a key tile for two sub-tiles (bf16 1.6 us at 128 wide,
    // 1.3 at 64; e4m3 2.0; with remainders half as much again), for one (1.3 us
    // at 128, the HBM's rate; 0.75 at 64; e4m3 1.5).  Against a block at 2.5
    // tiles of one cost for both types: five e4m3 windows 73.5 -> 66 us then, a
    // prompt of 8192 429 -> 422 us.
    const bool small = static_cast<long long>(p.max_window) * p.group <= kStackRows;
    AttendParams q = p;
    q.cost_block = 35;
    q.cost_pair = (D == 128 ? 16 : 12) + (E4M3 ? 4 : 0);
    q.cost_twice = q.cost_pair * 3 / 2;
    q.cost_stream = (D == 128 ? 13 : 8) + (E4M3 ? 3 : 0);
    return small ? launch_one<D, E4M3, true>(q, ws, s) : launch_one<D, E4M3, false>(q, ws, s);
}

cudaError_t launch_attend(const AttendParams& p, void* ws, cudaStream_t s) {
    if (p.c.D == 64) return p.c.e4m3 ? launch_form<64, true>(p, ws, s) : launch_form<64, false>(p, ws, s);
    return p.c.e4m3 ? launch_form<128, true>(p, ws, s) : launch_form<128, false>(p, ws, s);
}

}  // namespace sdm
