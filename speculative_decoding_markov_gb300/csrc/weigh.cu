// weigh.cu - the attention weight that every cached token got from a call's
// committed rows, added to what it had, on the tcgen05 tensor cores.
//
// Mathematics, for token j of a request and kv head g:
//     out_j = (j < ctx ? in_j : 0) + sum over rows p and heads h of g with j
//             visible of exp(scale q_ph . k_j - lse_ph)
// with the log-sum-exp that the attention left.  No maximum is needed: every
// term is a softmax weight, at most 1.
//
// Layout.  A product's 128 lanes are keys, its columns the query rows of one kv
// head (heads side by side, token by token): S = K Q^T.  A thread then owns a
// key, its sum over the columns never leaves its registers, a column's -lse is
// a broadcast read, and no result depends on an order of arrival.
//
// Work.  A unit is 256 keys of one request and kv head, a tile of 128 for each
// of two warpgroups, which share every tile of query rows.  Units laid end to
// end are cut into shares of equal cost, one per CTA (one CTA per SM).  If all
// rows of a head fit one tile (SMALL: decoding, verification), a cut never
// splits a unit, and the rows stay in shared memory while the keys of their
// head go by.  Else shares are cut between tiles of rows: the parts of a unit
// leave their sums in the workspace, and weigh_join_kernel adds them in order.
//
// A CTA: a warp walks the share, hands units out and loads keys page by page by
// TMA; one brings the query rows (by TMA, or gathered along a path; six split
// those of an e4m3 cache); one their -lse; one issues the products; eight, or 16
// unless SMALL, turn S into weights.
//
// An e4m3 cache: if SMALL its codes are operands as they are.  A bf16 query
// splits exactly into three e5m2 numbers (8 significant bits as 3 + 3 + 2,
// under a power of two per row that puts its largest element below 2^15;
// elements 2^24 smaller than that lose bits, at most 2^-31 of it), so S is
// three products over the same codes, and the scales of row and key follow in
// fp32.  Else, where a tile of keys meets many rows, its warpgroup turns the
// codes into bf16 once.
//
// Unless SMALL the keys of a unit stand in tensor memory: with both operands in
// shared memory a 128 x 128 x 128 product takes its whole bandwidth.
//
// What bounds it (32 query heads on 8 kv heads of 128, bf16, unless said):
//   64 windows of 1 to 8 tokens over 300 to 8000: HBM, 5.5 TB/s of keys (56 us).
//   A prompt of 8192 tokens: 224 us, 1.23 PFLOP/s.  Tensor pipe 52 %, the
//   exponentials' unit 53 %, issue 56 %: the products by themselves take 164 us
//   (without the weights) and the exponentials 122 us.  Tensor memory has three
//   buffers of scores for four groups of warps.
//   Two rows over 150001 to 199999, e4m3 (28 heads on 4): 50 us, 3.6 TB/s.  A
//   unit of 33 KB takes each of walker, products and weights about a
//   microsecond of waits and instructions (without its loads: 49 us; with a
//   third of the products 46; without sums 47; two groups of weight warps in
//   turn: 52, for want of registers).
//   One token over 500 keys: 5.7 us in a graph, the chain of plan, loads and
//   product.
#include <cudaTypedefs.h>

#include <algorithm>

#include "paged.cuh"

namespace sdm {
namespace {

constexpr int kTile = 128;            // keys of a tile, query rows of a tile
constexpr int kUnit = 2 * kTile;      // keys of a unit
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMostL = 3.4028235e38f;   // of -lse log2 e, where an lse is near the type's lowest value
constexpr int kTmemCols = 512;        // S buffers of 128 columns from 0; the tiles of keys (unless SMALL) at kTmemK
constexpr int kTmemK = 384;
constexpr int kHeavy = 6, kBase = 2;  // costs: a unit with a product if SMALL (1 without); a unit beside its row tiles
constexpr int kSpan = 64;             // units without a product that are handed out as one (SMALL: q1 of them)
constexpr int kExpStages = 16;        // e4m3 exponents of tiles

// A request's counted rows: window positions 0 .. n - 1 of its path (packed
// rows row0 .. row0 + wide - 1 hold its window) at tokens ctx, ctx + 1, ....
struct Counted {
    int row0, wide, n, ctx, bad;
};

__device__ __forceinline__ Counted counted_of(const WeighParams& p, int i) {
    Counted r;
    const long long tokens = min(table_tokens(p.c), static_cast<long long>(p.stride));
    const Window w = window_of(p.cu, nullptr, i, p.rows, 0x7fffffff, kMaxTokens);
    r.row0 = w.row0;
    r.wide = w.n;
    r.bad = w.bad;
    r.n = p.count ? __ldg(p.count + i) : w.n;
    r.ctx = __ldg(p.ctx + i);
    if (r.n < 0 || r.n > p.max_count || (r.n > w.n && !p.path) || r.ctx < 0) {
        r.bad |= SDM_DEV_BAD_WINDOW;
        r.n = min(max(r.n, 0), p.max_count);
        if (!p.path) r.n = min(r.n, w.n);
        r.ctx = max(r.ctx, 0);
    }
    if (static_cast<long long>(r.ctx) + r.n > tokens) {
        r.bad |= SDM_DEV_BAD_PAGE;
        r.ctx = static_cast<int>(min(static_cast<long long>(r.ctx), tokens));
        r.n = static_cast<int>(min(static_cast<long long>(r.n), tokens - r.ctx));
    }
    return r;
}

// The packed row of a counted one, or -1.
__device__ __forceinline__ long long row_of(const WeighParams& p, const Counted& w, int i, int wp) {
    const int off = p.path ? __ldg(p.path + static_cast<size_t>(i) * p.path_stride + wp) : wp;
    return static_cast<unsigned>(off) < static_cast<unsigned>(w.wide) ? w.row0 + off : -1;
}

// One unit, or the part of it that a CTA has.
struct __align__(16) Blk {
    int i, g, row0, wide;             // request, kv head, its window's packed rows
    int ctx, n, M, k0;                // committed tokens, all tokens, rows, first key
    int q0, q1, tiles, flags;         // tiles of rows q0 .. q1 - 1; tiles of keys (0: no more units)
};
enum { U_NEWQ = 1, U_FIRST = 2, U_LAST = 4, U_HAS = 8 };   // U_HAS: something is visible in it

template <int D, bool E4M3, bool SMALL>
struct Cfg {
    static constexpr bool kPlanes = E4M3 && SMALL;
    static constexpr int kKBytes = kTile * (kPlanes ? D : 2 * D);
    static constexpr int kPlane = kTile * D;                   // one e5m2 plane of a tile of rows
    static constexpr int kQBytes = kPlanes ? 3 * kPlane : kTile * 2 * D;
    // warps of the weights: one per scheduler hides little of the exponentials'
    // and the loads' latency, so many rows get two for each tile of keys
    static constexpr int kSoft = SMALL ? 8 : 16;
    // warps of the query rows and their -lse: two take longer to split a head's
    // rows into planes than its keys take (64 windows over 300 to 8000, e4m3: of
    // 1 to 8 tokens 103 us with two, 73 with six; of 16 to 30 tokens 302 and 159);
    // 16 warps in all leave a thread 128 registers, 18 only 96
    static constexpr int kRows = kPlanes ? 6 : 2;
    static constexpr int kThreads = 32 * (kSoft + 2 + kRows);
    static constexpr int kQSlots = SMALL ? 2 : D == 128 ? 4 : 8;
    static constexpr int kLStages = SMALL ? 2 : 4;
    static_assert(kLStages % 2 == 0, "a stage of -lse is always the same half's");
    static constexpr int kRing = SMALL ? 8 : 4;                // units handed out ahead
    static constexpr int kS = SMALL ? 4 : 3;                   // S buffers, products in turn
    static constexpr int kMiscBytes = kRing * sizeof(Blk) + kLStages * (kTile * 4 + 16) + (kPlanes ? 2 * kTile * 4 : 0) +
                                      (kPlanes ? kExpStages * kTile : 0) + (SMALL ? 0 : 2 * kUnit * 4) + 832;
    static constexpr int kFit = (232448 - kMiscBytes - kQSlots * kQBytes) / kKBytes;
    static constexpr int kKSlots = !SMALL ? 2 : kFit < 10 ? kFit : 10;
    static_assert(kFit >= (SMALL ? 4 : 2), "shared memory");
    static constexpr int kQ = kKSlots * kKBytes;
    static constexpr int kL = kQ + kQSlots * kQBytes;          // -lse log2 e of a tile's columns
    static_assert(kL >= 16384 * 8, "the plan's costs of up to 16384 requests");
    static constexpr int kCf = kL + kLStages * kTile * 4;      // planes: the columns' scales
    static constexpr int kExps = kCf + (kPlanes ? 2 * kTile * 4 : 0);
    static constexpr int kBlks = kExps + (kPlanes ? kExpStages * kTile : 0);
    static constexpr int kXch = kBlks + kRing * static_cast<int>(sizeof(Blk));   // sums of the second half's warps
    static constexpr int kBars = kXch + (SMALL ? 0 : 2 * kUnit * 4);
};

template <int K, int Q, int L, int U, int S>
struct Bars {
    uint64_t k_full[K], k_empty[K], q_full[Q], q_empty[Q], l_full[L], l_empty[L];
    // A buffer is filled for one of two or four groups of warps (tile of keys,
    // half), and a parity tells only the last phase from the next: each has a
    // barrier of its own for it.
    uint64_t s_full[S][4], s_empty[S], kt_full[2], k_idle[2], j_full[2][2], j_empty[2][2], blk_full[U], blk_empty[U], x_full[kExpStages];
    uint64_t drain;
    uint32_t live[L][5];              // columns of the stage that add something; whether some do not
    uint32_t tmem;
};

// What a share's ends leave for weigh_join_kernel.
struct Part {
    int rest;                         // the share starts a unit and does not finish it
    int head;                         // its first part continues a unit: 0 no, 1 and finishes it, 2 and does not
    int i, g, k0, n, ctx, pad;        // the started unit
};
struct Scratch {
    Part* part;                       // [grid]
    float* sum;                       // [grid][2][kUnit]: what continues a unit, what starts one
};

// ---------------------------------------------------------------------------
// A request's units and their costs
// ---------------------------------------------------------------------------
struct Req {
    Counted w;
    int n, M, QT, units;              // tokens, rows, tiles of rows, units of a head
    int us, ul;                       // units below us or from ul on have a product (SMALL)
};

__device__ __forceinline__ Req req_of(const WeighParams& p, int i) {
    Req r;
    r.w = counted_of(p, i);
    r.n = r.w.ctx + r.w.n;
    r.M = r.w.n * p.group;
    r.QT = (r.M + p.sub - 1) / p.sub;
    r.units = (r.n + kUnit - 1) / kUnit;
    r.us = r.ul = r.units;
    if (r.M == 0) {
        r.us = 0;
        r.ul = r.units;
    } else if (p.window > 0) {
        r.us = min(r.units, static_cast<int>((static_cast<long long>(p.sinks) + kUnit - 1) / kUnit));
        r.ul = min(r.units, max(0, r.w.ctx + 1 - p.window) / kUnit);
        r.ul = max(r.ul, r.us);
    }
    return r;
}

// Tiles of rows [q0, q1) that see some key of a unit.
__device__ __forceinline__ void rows_of(const WeighParams& p, const Req& r, int u, int& q0, int& q1) {
    const int k0 = u * kUnit;
    q0 = k0 > r.w.ctx ? (k0 - r.w.ctx) * p.group / p.sub : 0;
    q1 = r.QT;
    if (p.window > 0 && k0 >= p.sinks) {
        const long long last = min(k0 + kUnit, r.n) - 1;       // seen by the rows below last - ctx + window
        const long long end = last - r.w.ctx + p.window;
        if (end < r.w.n) q1 = end <= 0 ? 0 : static_cast<int>((end * p.group + p.sub - 1) / p.sub);
    }
    q1 = max(q0, q1);
}

template <bool SMALL>
__device__ __forceinline__ int cost_of(const WeighParams& p, const Req& r, int u) {
    if (SMALL) return u < r.us || u >= r.ul ? kHeavy : 1;
    int q0, q1;
    rows_of(p, r, u, q0, q1);
    return kBase + q1 - q0;
}

// Cost of a head's units 0 .. u - 1 (SMALL).
__device__ __forceinline__ long long before_unit(const Req& r, int u) {
    return static_cast<long long>(min(u, r.us) + max(0, u - r.ul)) * kHeavy + min(max(u - r.us, 0), r.ul - r.us);
}

// Where a CTA's share starts: the unit in which its first cost unit lies.
struct Start {
    unsigned long long us, u0, u1;    // cost at which that unit begins, the share [u0, u1)
    int i, g, u, pad;
};

// The unit of a head that cost `into` of it lies in (SMALL).
__device__ __forceinline__ int unit_at(int us, int ul, unsigned long long into) {
    const unsigned long long first = static_cast<unsigned long long>(us) * kHeavy, mid = first + (ul - us);
    if (into < first) return static_cast<int>(into / kHeavy);
    if (into < mid) return us + static_cast<int>(into - first);
    return ul + static_cast<int>((into - mid) / kHeavy);
}

__device__ __forceinline__ void share_of(unsigned long long total, unsigned long long& u0, unsigned long long& u1) {
    const unsigned long long each = total >> 32 ? total / gridDim.x : static_cast<unsigned>(total) / gridDim.x;
    const unsigned more = static_cast<unsigned>(total - each * gridDim.x);
    u0 = each * blockIdx.x + min(blockIdx.x, more);
    u1 = u0 + each + (blockIdx.x < more ? 1 : 0);
}

// Where the share starts, for at most 32 requests (SMALL): by the walking warp
// alone, a lane per request, while the others set themselves up.
__device__ __forceinline__ Start plan_few(const WeighParams& p) {
    const int lane = threadIdx.x & 31;
    Req r = {};
    if (lane < p.R) r = req_of(p, lane);
    if (r.w.bad && blockIdx.x == 0) set_status(p.dev_status, r.w.bad);
    const unsigned long long head = before_unit(r, r.units), mine = head * p.c.heads;
    unsigned long long sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
    }
    Start st = {};
    share_of(__shfl_sync(0xffffffffu, sum, 31), st.u0, st.u1);
    const unsigned hit = __ballot_sync(0xffffffffu, sum > st.u0);
    const int k = hit ? __ffs(hit) - 1 : 0;
    const unsigned long long c = max(__shfl_sync(0xffffffffu, head, k), 1ull);
    const int us = __shfl_sync(0xffffffffu, r.us, k), ul = __shfl_sync(0xffffffffu, r.ul, k);
    st.us = __shfl_sync(0xffffffffu, sum - mine, k);
    unsigned long long into = st.u0 - st.us;
    st.i = k;
    st.g = into >> 32 || c >> 32 ? static_cast<int>(into / c) : static_cast<unsigned>(into) / static_cast<unsigned>(c);
    into -= st.g * c;
    st.u = unit_at(us, ul, into);
    st.us += st.g * c + static_cast<unsigned long long>(min(st.u, us) + max(0, st.u - ul)) * kHeavy +
             min(max(st.u - us, 0), ul - us);
    return st;
}

// cost: shared memory for R entries.  By all warps.
template <bool SMALL, int kThreads>
__device__ __forceinline__ void plan(const WeighParams& p, unsigned long long* cost, unsigned long long* wsum,
                                     Start* start) {
    constexpr int kWarps = kThreads / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (SMALL) {
        for (int i = tid; i < p.R; i += kThreads) {
            const Req r = req_of(p, i);
            if (r.w.bad && blockIdx.x == 0) set_status(p.dev_status, r.w.bad);
            cost[i] = before_unit(r, r.units) * p.c.heads;
        }
    } else {
        for (int i = warp; i < p.R; i += kWarps) {
            const Req r = req_of(p, i);
            if (r.w.bad && blockIdx.x == 0 && lane == 0) set_status(p.dev_status, r.w.bad);
            unsigned long long c = 0;
            for (int u = lane; u < r.units; u += 32) c += cost_of<false>(p, r, u);
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
        const unsigned long long v = __shfl_up_sync(0xffffffffu, incl, o);
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
        const Req r = req_of(p, i);
        const unsigned long long c = cost[i] / p.c.heads;      // of a head; not 0, for the share's start lies in it
        unsigned long long into = u0 - start->us;
        const int g = static_cast<int>(into / c);
        unsigned long long us = start->us + g * c;
        into -= g * c;
        int u = 0;
        if (SMALL) {
            u = unit_at(r.us, r.ul, into);
            us += before_unit(r, u);
        } else {
            for (int u0_ = 0; u0_ < r.units; u0_ += 32) {
                const unsigned long long one = u0_ + lane < r.units ? cost_of<false>(p, r, u0_ + lane) : 0;
                unsigned long long sum = one;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const unsigned long long v = __shfl_up_sync(0xffffffffu, sum, o);
                    if (lane >= o) sum += v;
                }
                const unsigned hit = __ballot_sync(0xffffffffu, sum > into);
                if (hit) {
                    const int at = __ffs(hit) - 1;
                    u = u0_ + at;
                    us += __shfl_sync(0xffffffffu, sum - one, at);
                    break;
                }
                const unsigned long long all = __shfl_sync(0xffffffffu, sum, 31);
                into -= all;
                us += all;
            }
        }
        __syncwarp();
        if (lane == 0) {
            start->g = g;
            start->u = u;
            start->us = us;
        }
    }
    fence_proxy_async_smem();   // `cost` lies where TMA is about to write
    __syncthreads();
}

__device__ __forceinline__ bool wait_or_fail(const WeighParams& p, uint64_t* bar, uint32_t parity) {
    if (__builtin_expect(__all_sync(0xffffffffu, mbar_try_wait(bar, parity)), 1)) return true;   // one answer a warp
    const uint64_t t0 = globaltimer();
#pragma unroll 1
    do {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    } while (__all_sync(0xffffffffu, globaltimer() - t0 < kWaitLimitNs));
    set_status(p.dev_status, SDM_DEV_TIMEOUT);
    return false;
}

// A place in a ring and the parity of the phase it is in.
template <int N>
struct Ring {
    int at = 0;
    uint32_t turn = 0;
    __device__ __forceinline__ void step() {
        if (++at == N) {
            at = 0;
            ++turn;
        }
    }
    __device__ __forceinline__ uint32_t full() const { return turn & 1; }           // for the reader
    __device__ __forceinline__ uint32_t empty() const { return (turn & 1) ^ 1; }    // for the writer: passes at first
};

// N (2 or 4) products along the rows' bytes, 32 bytes a step, in one statement:
// the lane elect.sync picks issues them with nothing but the descriptors' steps
// between (one statement each: 930 clocks for the eight of a tile).
template <bool F8, int N>
__device__ __forceinline__ void issue(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add) {
#define SDM_MMA4(KIND)                                                                                             \
    asm volatile(                                                                                                  \
        "{\n\t.reg .pred e, p, q;\n\t.reg .b64 a, b;\n\telect.sync _|e, 0xffffffff;\n\t"                         \
        "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 q, 0, 0;\n\t"                                                        \
        "@e tcgen05.mma.cta_group::1.kind::" KIND " [%0], %1, %2, %3, p;\n\t"                                      \
        "add.s64 a, %1, 2;\n\tadd.s64 b, %2, 2;\n\t"                                                               \
        "@e tcgen05.mma.cta_group::1.kind::" KIND " [%0], a, b, %3, q;\n\t"                                        \
        "add.s64 a, %1, 4;\n\tadd.s64 b, %2, 4;\n\t"                                                               \
        "@e tcgen05.mma.cta_group::1.kind::" KIND " [%0], a, b, %3, q;\n\t"                                        \
        "add.s64 a, %1, 6;\n\tadd.s64 b, %2, 6;\n\t"                                                               \
        "@e tcgen05.mma.cta_group::1.kind::" KIND " [%0], a, b, %3, q;\n\t}" ::"r"(d),                             \
        "l"(a), "l"(b), "r"(idesc), "r"(add)                                                                       \
        : "memory")
    static_assert(N == 4 || (N == 2 && F8), "steps");
    if constexpr (!F8) {
        SDM_MMA4("f16");
    } else if constexpr (N == 4) {
        SDM_MMA4("f8f6f4");
    } else {
        asm volatile(
            "{\n\t.reg .pred e, p, q;\n\t.reg .b64 a, b;\n\telect.sync _|e, 0xffffffff;\n\t"
            "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 q, 0, 0;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t"
            "add.s64 a, %1, 2;\n\tadd.s64 b, %2, 2;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, q;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(add)
            : "memory");
    }
#undef SDM_MMA4
}

// The same four bf16 products with A in tensor memory, 8 columns a step.
__device__ __forceinline__ void issue_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred e, p, q;\n\t.reg .b64 b;\n\t.reg .b32 a;\n\telect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 q, 0, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
        "add.s32 a, %1, 8;\n\tadd.s64 b, %2, 2;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, q;\n\t"
        "add.s32 a, %1, 16;\n\tadd.s64 b, %2, 4;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, q;\n\t"
        "add.s32 a, %1, 24;\n\tadd.s64 b, %2, 6;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, q;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
}

// kind::f8f6f4: e4m3 A (0 at bit 7), e5m2 B (1 at bit 10), fp32 accumulator
__device__ __forceinline__ uint32_t idesc_f8(int M, int N) {
    return (1u << 4) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// Descriptor of 64-byte rows, 64-byte swizzle (mode 4).
__device__ __forceinline__ uint64_t smem_desc_sw64(uint32_t saddr) {
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (1ull << 16) | (static_cast<uint64_t>(512 >> 4) << 32) |
           (1ull << 46) | (4ull << 61);
}

__device__ __forceinline__ uint32_t f32x2_to_e5m2x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 e5m2x2_to_f32x2(uint32_t codes) {
    uint32_t r;
    asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(codes)));
    return f16x2_to_f32x2(r);
}

__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y), "f"(z.x), "f"(z.y));
    return r;
}
__device__ __forceinline__ float2 mul2(float2 x, float2 y) {
    float2 r;
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmul.rn.f32x2 a, a, b;\n\t"
        "mov.b64 {%0, %1}, a;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
    return r;
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
    float2 r;
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 a, a, b;\n\t"
        "mov.b64 {%0, %1}, a;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
    return r;
}

// Adds the weights of N columns: 2^(c f x + l), f the columns' scales (planes),
// l their -lse log2 e.  A scale of at most 1 comes before c, so that nothing on
// the way is larger than the score; BIG: one above 1 after it.
template <bool PLANES, bool BIG, int N>
__device__ __forceinline__ void add_weights(const uint32_t (&x)[N], float c, const float4* l4, const float4* f4,
                                            float2 (&acc)[4]) {
    const float2 cc = make_float2(c, c);
#pragma unroll
    for (int k = 0; k < N / 4; ++k) {
        const float4 l = l4[k];
        float2 a = make_float2(__uint_as_float(x[4 * k]), __uint_as_float(x[4 * k + 1]));
        float2 b = make_float2(__uint_as_float(x[4 * k + 2]), __uint_as_float(x[4 * k + 3]));
        if constexpr (PLANES) {
            const float4 f = f4[k];
            if constexpr (BIG) {
                a = mul2(mul2(a, make_float2(fminf(f.x, 1.f), fminf(f.y, 1.f))), cc);
                b = mul2(mul2(b, make_float2(fminf(f.z, 1.f), fminf(f.w, 1.f))), cc);
                a = fma2(a, make_float2(fmaxf(f.x, 1.f), fmaxf(f.y, 1.f)), make_float2(l.x, l.y));
                b = fma2(b, make_float2(fmaxf(f.z, 1.f), fmaxf(f.w, 1.f)), make_float2(l.z, l.w));
            } else {
                a = fma2(mul2(a, make_float2(f.x, f.y)), cc, make_float2(l.x, l.y));
                b = fma2(mul2(b, make_float2(f.z, f.w)), cc, make_float2(l.z, l.w));
            }
        } else {
            a = fma2(a, cc, make_float2(l.x, l.y));
            b = fma2(b, cc, make_float2(l.z, l.w));
        }
        acc[2 * (k & 1)] = add2(acc[2 * (k & 1)], make_float2(fast_exp2(a.x), fast_exp2(a.y)));
        acc[2 * (k & 1) + 1] = add2(acc[2 * (k & 1) + 1], make_float2(fast_exp2(b.x), fast_exp2(b.y)));
    }
}

// Scores of columns that a key is not seen by become -infinity (whose weight is
// 0 whatever their l, which is no NaN and not +infinity): all but lo .. hi - 1,
// and those whose bit is not set in `live`.
template <int N>
__device__ __forceinline__ void hide(uint32_t (&x)[N], int lo, int hi, uint32_t live) {
    const int from = max(lo, 0);
    live &= (from >= 32 ? 0u : ~0u << from) & (hi >= 32 ? ~0u : hi <= 0 ? 0u : (1u << hi) - 1u);
#pragma unroll
    for (int k = 0; k < N; ++k) x[k] = (live >> k) & 1u ? x[k] : 0xff800000u;
}

// The same of a tile's `cols` columns, from tensor memory, some of whose scales
// are above 1.  Not inline: the registers that it takes would cost the others'
// form a fifth of its time (two contexts of 150001 to 199999: 63.7 us, 51.2 so).
__device__ __noinline__ float add_big(uint32_t s_at, int cols, int lo, int hi, const uint32_t* live, float c,
                                      const float4* l4, const float4* f4) {
    float2 acc[4] = {};
    uint32_t x[16];
#pragma unroll 1
    for (int at = 0; at < cols; at += 16) {
        tmem_ld16(s_at + at, x);
        tmem_ld_wait();
        hide(x, lo - at, hi - at, live[at / 32] >> (at & 31));
        add_weights<true, true>(x, c, l4 + at / 4, f4 + at / 4, acc);
    }
    const float2 two = add2(add2(acc[0], acc[1]), add2(acc[2], acc[3]));
    return two.x + two.y;
}

// ---------------------------------------------------------------------------
// The kernel
// ---------------------------------------------------------------------------
template <int D, bool E4M3, bool SMALL>
__global__ void __launch_bounds__(Cfg<D, E4M3, SMALL>::kThreads, 1)
    weigh_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmQ,
                 const __grid_constant__ WeighParams p, const __grid_constant__ Scratch ws) {
    using C = Cfg<D, E4M3, SMALL>;
    constexpr bool kPlanes = C::kPlanes;
    constexpr int kSoft = C::kSoft;
    using B = Bars<C::kKSlots, C::kQSlots, C::kLStages, C::kRing, C::kS>;
    static_assert(C::kBars + sizeof(B) <= 232448, "shared memory");
    extern __shared__ __align__(1024) uint8_t smem[];
    B& bar = *reinterpret_cast<B*>(smem + C::kBars);
    Blk* blks = reinterpret_cast<Blk*>(smem + C::kBlks);
    float* l2 = reinterpret_cast<float*>(smem + C::kL);
    float* cf = reinterpret_cast<float*>(smem + C::kCf);
    Start* start = reinterpret_cast<Start*>(smem + C::kL);     // only until the roles begin
    unsigned long long* wsum = reinterpret_cast<unsigned long long*>(smem + C::kL + 64);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (warp == kSoft) {
        if (lane == 0) {
            tma_prefetch_desc(&tmK);
            tma_prefetch_desc(&tmQ);
        }
    } else if (warp == kSoft + 1) {
        tmem_alloc(&bar.tmem, kTmemCols);
        tmem_relinquish();
    } else if (warp == kSoft + 2) {
        for (int k = lane; k < C::kKSlots; k += 32) {
            mbar_init(&bar.k_full[k], 1);
            mbar_init(&bar.k_empty[k], 1);
        }
        if (lane < C::kQSlots) {
            mbar_init(&bar.q_full[lane], SMALL ? C::kRows : 1);
            mbar_init(&bar.q_empty[lane], SMALL ? 9 : 1);
        }
        if (lane < C::kLStages) {
            mbar_init(&bar.l_full[lane], 1);
            mbar_init(&bar.l_empty[lane], 8);
        }
        if (lane < C::kS) {
            for (int k = 0; k < 4; ++k) mbar_init(&bar.s_full[lane][k], 1);
            mbar_init(&bar.s_empty[lane], 4);
        }
        if (lane < 2) {
            mbar_init(&bar.kt_full[lane], D == 128 ? 8 : 4);
            mbar_init(&bar.k_idle[lane], 1);
        }
        if (lane < 4) {
            mbar_init(&bar.j_full[0][0] + lane, 4);
            mbar_init(&bar.j_empty[0][0] + lane, 4);
        }
        if (lane < C::kRing) {
            mbar_init(&bar.blk_full[lane], 1);
            mbar_init(&bar.blk_empty[lane], kSoft + 1 + C::kRows);   // the warps that read it
        }
        if (lane < kExpStages) {
            mbar_init(&bar.x_full[lane], 1);
        }
        if (lane == 0) mbar_init(&bar.drain, 1);
        fence_mbar_init();
    }
    pdl_wait();
    pdl_trigger();
    const bool few = SMALL && p.R <= 32;
    if (!few) plan<SMALL, C::kThreads>(p, reinterpret_cast<unsigned long long*>(smem), wsum, start);
    Start st = *start;                // read before the roles use its place
    // rows of a tile that no query row fills are zeros, so that their columns are finite
    for (int k = tid; k < C::kQSlots * C::kQBytes / 16; k += C::kThreads)
        reinterpret_cast<uint4*>(smem + C::kQ)[k] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar.tmem;

    Ring<C::kRing> rd;
    // waits for the next unit; false at the end (or with ok false)
    auto take = [&](bool& ok, Blk& b) {
        ok = wait_or_fail(p, &bar.blk_full[rd.at], rd.full());
        if (!ok) return false;
        const int4* src = reinterpret_cast<const int4*>(blks + rd.at);
        int4* dst = reinterpret_cast<int4*>(&b);
#pragma unroll
        for (int k = 0; k < static_cast<int>(sizeof(Blk) / 16); ++k) dst[k] = src[k];
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.blk_empty[rd.at]);
        rd.step();
        return b.tiles > 0;
    };

    if (warp == kSoft) {
        // ------------------------------------------------------------------
        // walker: the share's units, and their keys
        // ------------------------------------------------------------------
        bool ok = true;
        if (few) st = plan_few(p);
        unsigned long long us = st.us;
        int i = st.i, g = st.g, u = st.u, have = -1, loaded_i = -1, loaded_g = -1;
        Req r;
        Ring<C::kRing> wr;
        Ring<C::kKSlots> kr, k_sent;      // the next place, and the one after the last that was filled
        Ring<kExpStages> xr, x_sent;
        bool live_share = st.u0 < st.u1;
        Part part = {};
        // page ids of a unit's keys, a lane per page, loaded a unit ahead: the
        // table's latency would else stand before every unit's first copy
        const int unit_pages = kUnit >> p.c.page_shift;
        auto page_at = [&](int i, int u) {
            const long long col = static_cast<long long>(u) * unit_pages + lane;
            return lane < unit_pages && col < p.c.max_pages ? __ldg(p.c.table + static_cast<size_t>(i) * p.c.max_pages + col) : -1;
        };
        int ahead = -1, ahead_i = -1, ahead_u = -1;
        while (ok) {
            Blk b = {};
            bool got = false;
            while (live_share && us < st.u1) {
                if (have != i) {
                    if (i >= p.R) break;
                    r = req_of(p, i);
                    have = i;
                }
                if (u >= r.units) {
                    u = 0;
                    if (++g >= p.c.heads) {
                        g = 0;
                        ++i;
                    }
                    continue;
                }
                int q0 = 0, q1 = 1, span = 1;
                const int cost = cost_of<SMALL>(p, r, u);
                b.flags = U_FIRST | U_LAST;
                bool mine;
                if (SMALL) {
                    mine = us >= st.u0;
                    if (cost == kHeavy) b.flags |= U_HAS;
                    else if (mine) q1 = span = static_cast<int>(min(static_cast<unsigned long long>(min(r.ul - u, kSpan)), st.u1 - us));
                } else {
                    rows_of(p, r, u, q0, q1);
                    const int all = q1 - q0;
                    if (all == 0) {
                        mine = us >= st.u0;
                    } else {
                        // tile k of the rows stands at cost us + kBase + k
                        const unsigned long long at = us + kBase;
                        const int t0 = st.u0 <= at ? 0 : static_cast<int>(min(st.u0 - at, static_cast<unsigned long long>(all)));
                        const int t1 = st.u1 <= at ? 0 : static_cast<int>(min(st.u1 - at, static_cast<unsigned long long>(all)));
                        mine = t1 > t0;
                        b.flags = U_HAS | (t0 == 0 ? U_FIRST : 0) | (t1 == all ? U_LAST : 0);
                        if (mine && t0 > 0) part.head = t1 == all ? 1 : 2;
                        if (mine && t0 == 0 && t1 < all) {
                            part.rest = 1;
                            part.i = i, part.g = g, part.k0 = u * kUnit, part.n = r.n, part.ctx = r.w.ctx;
                        }
                        q1 = q0 + t1;
                        q0 += t0;
                    }
                }
                b.i = i, b.g = g, b.row0 = r.w.row0, b.wide = r.w.wide;
                b.ctx = r.w.ctx, b.n = r.n, b.M = r.M, b.k0 = u * kUnit;
                b.q0 = q0, b.q1 = q1;
                b.tiles = r.n - b.k0 > kTile ? 2 : 1;
                us += static_cast<unsigned>(cost * span);
                u += span;
                if (mine) {
                    got = true;
                    break;
                }
            }
            if (!got) b.tiles = 0;
            if (got && (b.flags & U_HAS) && (loaded_i != b.i || loaded_g != b.g)) {
                b.flags |= U_NEWQ;
                loaded_i = b.i;
                loaded_g = b.g;
            }
            ok = wait_or_fail(p, &bar.blk_empty[wr.at], wr.empty());
            if (!ok) break;
            if (lane == 0) {
                blks[wr.at] = b;
                mbar_arrive(&bar.blk_full[wr.at]);
            }
            wr.step();
            if (!got) break;
            if (!(b.flags & U_HAS) || (E4M3 && !SMALL)) continue;
            // its keys, a lane per page
            const int pages = kTile >> p.c.page_shift, page = 1 << p.c.page_shift;
            const int this_u = b.k0 / kUnit;
            const int ids = ahead_i == b.i && ahead_u == this_u ? ahead : page_at(b.i, this_u);
            ahead_i = b.i;
            ahead_u = this_u + 1;
            ahead = page_at(ahead_i, ahead_u);
            // both tiles at once: lanes 0 .. 15 the first one's pages, 16 .. 31 the second's
            const int t = lane >> 4, l = lane & 15;
            const int live = min(pages, (b.n - b.k0 - t * kTile + page - 1) >> p.c.page_shift);   // negative: no second one
            int pg = __shfl_sync(0xffffffffu, ids, (t * pages + l) & 31);
            if (l < live && static_cast<unsigned>(pg) >= static_cast<unsigned>(p.c.n_pages)) {
                set_status(p.dev_status, SDM_DEV_BAD_PAGE);
                pg = 0;
            }
            const int y = (pg * p.c.heads + b.g) << p.c.page_shift;
            int slot = kr.at, stage = xr.at;
            for (int k = 0; k < b.tiles && ok; ++k) {
                ok = wait_or_fail(p, &bar.k_empty[kr.at], kr.empty());
                if (!ok) break;
                if (t == k) slot = kr.at, stage = xr.at;
                kr.step();
                // The exponents' stages are not waited for: a tile's keys wait for
                // the product kKSlots before it, which waits for the weights kS
                // before that, by when these have read theirs.
                static_assert(!kPlanes || C::kKSlots + C::kS + 2 <= kExpStages, "stages of exponents");
                xr.step();
            }
            if (!ok) break;
            if (l < (kPlanes ? 2 : 1) && t < b.tiles)
                mbar_arrive_expect_tx(l == 0 ? &bar.k_full[slot] : &bar.x_full[stage],
                                      static_cast<uint32_t>(live) * page * (l == 1 ? 1 : kPlanes ? D : 2 * D));
            __syncwarp();
            if (l < live) {
                uint8_t* to = smem + slot * C::kKBytes;
                if constexpr (kPlanes) {
                    tma_load_2d(to + l * page * D, &tmK, &bar.k_full[slot], 0, y);
                    bulk_load(smem + C::kExps + stage * kTile + l * page, p.c.k_exp + y, page, &bar.x_full[stage]);
                } else {
#pragma unroll
                    for (int h = 0; h < D / 64; ++h)
                        tma_load_2d(to + h * (kTile * 128) + l * page * 128, &tmK, &bar.k_full[slot], h * 64, y);
                }
            }
            __syncwarp();
            k_sent = kr;
            x_sent = xr;
        }
        if (!SMALL && lane == 0) ws.part[blockIdx.x] = part;
        if (!ok) {
            // copies in flight land before the CTA may exit
            for (int k = 0; k < C::kKSlots; ++k)
                if (k_sent.turn > 0 || k < k_sent.at)
                    mbar_wait(&bar.k_full[k], k < k_sent.at ? k_sent.turn & 1 : (k_sent.turn & 1) ^ 1);
            if (kPlanes)
                for (int k = 0; k < kExpStages; ++k)
                    if (x_sent.turn > 0 || k < x_sent.at)
                        mbar_wait(&bar.x_full[k], k < x_sent.at ? x_sent.turn & 1 : (x_sent.turn & 1) ^ 1);
        }
    } else if (warp == kSoft + 1) {
        // ------------------------------------------------------------------
        // products
        // ------------------------------------------------------------------
        bool ok = true;
        Ring<C::kKSlots> kr;
        Ring<C::kQSlots> qr;          // SMALL: the slot in use
        Ring<C::kS> sr;
        bool any_q = false;
        uint32_t n_units = 0, n_two = 0, n_q = 0;   // units, those of two tiles, tiles of rows
        Blk b;
        while (take(ok, b)) {
            if (!(b.flags & U_HAS)) continue;
            if (SMALL && (b.flags & U_NEWQ)) {
                if (any_q) {
                    mma_commit_warp(&bar.q_empty[qr.at]);
                    qr.step();
                }
                any_q = true;
                ok = wait_or_fail(p, &bar.q_full[qr.at], qr.full());
                if (!ok) break;
            }
            if constexpr (!SMALL) {
                // the unit's keys into tensor memory, once the products of the
                // one before have read theirs (for e4m3 the warpgroups do it)
                if constexpr (!E4M3) {
                    if (n_units > 0) {
                        mma_commit_warp(&bar.k_idle[0]);
                        ok = wait_or_fail(p, &bar.k_idle[0], (n_units - 1) & 1);
                    }
                    for (int t = 0; t < b.tiles && ok; ++t) {
                        ok = wait_or_fail(p, &bar.k_full[kr.at], kr.full());
                        if (!ok) break;
                        const uint64_t a = smem_desc_sw128(smem_u32(smem + kr.at * C::kKBytes), 16, 1024);
#pragma unroll
                        for (int k = 0; k < D / 16; ++k)
                            tmem_cp_128x256b_warp(tmem + kTmemK + t * (D / 2) + k * 8,
                                                  a + (k / 4) * ((kTile * 128) >> 4) + (k % 4) * 2);
                        mma_commit_warp(&bar.k_empty[kr.at]);
                        kr.step();
                    }
                } else {
                    for (int t = 0; t < b.tiles && ok; ++t) ok = wait_or_fail(p, &bar.kt_full[t], t == 0 ? n_units & 1 : n_two & 1);
                    n_two += b.tiles == 2;
                }
                ++n_units;
                if (!ok) break;
            }
            for (int q = b.q0; q < b.q1 && ok; ++q) {
                if (!SMALL) ok = wait_or_fail(p, &bar.q_full[qr.at], qr.full());
                const int N = !SMALL ? kTile : b.M <= 16 ? 16 : (b.M + 31) & ~31;   // what the weights read
                for (int t = 0; t < b.tiles && ok; ++t) {
                    if (SMALL) ok = wait_or_fail(p, &bar.k_full[kr.at], kr.full());
                    if (ok) ok = wait_or_fail(p, &bar.s_empty[sr.at], sr.empty());
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t d = tmem + sr.at * 128;
                    const uint32_t ka = smem_u32(smem + kr.at * C::kKBytes), qa = smem_u32(smem + C::kQ + qr.at * C::kQBytes);
                    if constexpr (kPlanes) {
                        const uint64_t a = D == 128 ? smem_desc_sw128(ka, 16, 1024) : smem_desc_sw64(ka);
                        const uint64_t q_ = D == 128 ? smem_desc_sw128(qa, 16, 1024) : smem_desc_sw64(qa);
                        const uint32_t id = idesc_f8(kTile, N);
#pragma unroll
                        for (int pl = 0; pl < 3; ++pl)
                            issue<true, D / 32>(d, a, q_ + ((pl * C::kPlane) >> 4), id, pl > 0);
                    } else {
                        const uint64_t q_ = smem_desc_sw128(qa, 16, 1024);
                        const uint32_t id = idesc_bf16_f32(kTile, N, false);
#pragma unroll
                        for (int h = 0; h < D / 64; ++h) {
                            const uint64_t panel = h * ((kTile * 128) >> 4);
                            if constexpr (SMALL) issue<false, 4>(d, smem_desc_sw128(ka, 16, 1024) + panel, q_ + panel, id, h > 0);
                            else issue_ts(d, tmem + kTmemK + t * (D / 2) + h * 32, q_ + panel, id, h > 0);
                        }
                    }
                    mma_commit_warp(&bar.s_full[sr.at][SMALL ? t : t + 2 * (n_q & 1)]);
                    sr.step();
                    if (SMALL) {
                        mma_commit_warp(&bar.k_empty[kr.at]);
                        kr.step();
                    }
                }
                ++n_q;
                if (!SMALL && ok) {
                    mma_commit_warp(&bar.q_empty[qr.at]);
                    qr.step();
                }
            }
            if (!ok) break;
            if constexpr (E4M3 && !SMALL)
                for (int t = 0; t < b.tiles; ++t) mma_commit_warp(&bar.k_idle[t]);
        }
        // products in flight end before the tensor memory goes
        mma_commit_warp(&bar.drain);
        mbar_wait(&bar.drain, 0);
    } else if (warp > kSoft + 1) {
        // ------------------------------------------------------------------
        // the query rows (one warp; split into planes: all of them) and their -lse
        // ------------------------------------------------------------------
        const bool rows_warp = warp != kSoft + 3;
        bool ok = true;
        Ring<C::kQSlots> qr;
        Ring<C::kLStages> lr;
        Blk b;
        int sent = 0;
        const int tokens = p.sub / p.group;   // of a tile
        // four columns a lane: window position in the tile, and head
        int col_wp[4], col_h[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            col_wp[k] = (k * 32 + lane) / p.group;
            col_h[k] = (k * 32 + lane) - col_wp[k] * p.group;
            if (k * 32 + lane >= p.sub) col_wp[k] = 1 << 30;
        }
        auto lse_of = [&](const Blk& b, int q, float (&z)[4]) {
            Counted w;
            w.row0 = b.row0;
            w.wide = b.wide;
            const int rows = b.M / p.group - q * tokens;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                z[k] = -INFINITY;
                if (col_wp[k] < rows) {
                    const long long row = row_of(p, w, b.i, q * tokens + col_wp[k]);
                    if (row >= 0) z[k] = __ldg(p.lse + row * p.H + b.g * p.group + col_h[k]);
                    else set_status(p.dev_status, SDM_DEV_BAD_WINDOW);
                }
            }
        };
        // -lse log2 e, -infinity for columns that add nothing, which are noted
        // (but for those behind a full tile's rows, where the scores are 0 or NaN)
        auto put_lse = [&](const Blk& b, int q, const float (&z)[4], float* to, uint32_t (&live)[5]) {
            const bool full = b.M - q * p.sub >= p.sub;
            uint32_t all = ~0u;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int col = k * 32 + lane;
                const bool adds = z[k] > -INFINITY;             // a NaN does not
                to[col] = adds ? fminf(-z[k] * kLog2e, kMostL) : -INFINITY;   // finite: see hide()
                const uint32_t bits = __ballot_sync(0xffffffffu, adds || (full && col >= p.sub));
                if (lane == 0) live[k] = bits;
                all &= bits;
            }
            if (lane == 0) live[4] = all != ~0u;
        };
        // rows of tile q of the head into a slot, 16 bytes at a time, zeros up to N
        auto gather = [&](const Blk& b, int q, uint8_t* slot) {
            constexpr int kChunks = D / 8, kPer = 32 / kChunks;   // 16-byte pieces of a row; rows of a step
            const int M = min(p.sub, b.M - q * p.sub), N = (M + 31) & ~31;
            Counted w;
            w.row0 = b.row0;
            w.wide = b.wide;
            const int c = lane % kChunks;
            int wp = (lane / kChunks) / p.group, h = (lane / kChunks) - wp * p.group;
            wp += q * tokens;
#pragma unroll 4
            for (int r = lane / kChunks; r < N; r += kPer) {
                const long long row = r < M ? row_of(p, w, b.i, wp) : -1;
                const uint16_t* src = p.q;
                if (row >= 0) src += row * p.q_stride + static_cast<size_t>(b.g * p.group + h) * D + c * 8;
                cp_async_16(slot + (c / 8) * (kTile * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4), src, row >= 0 ? 16 : 0);
                h += kPer;
                while (h >= p.group) {
                    h -= p.group;
                    ++wp;
                }
            }
            cp_async_wait_all();
            fence_proxy_async_smem();
            __syncwarp();
        };
        // the same as three planes of e5m2, and the rows' scales: this warp's groups of 4 rows
        auto split = [&](const Blk& b, uint8_t* slot, float* scale) {
            constexpr int kPer = D / 32;   // elements of a lane
            const int M = b.M, N = (M + 31) & ~31;
            Counted w;
            w.row0 = b.row0;
            w.wide = b.wide;
            for (int r0 = 4 * (warp - kSoft - 2); r0 < N; r0 += 4 * C::kRows) {
                uint32_t x[4][2];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int m = r0 + e;
                    x[e][0] = x[e][1] = 0;
                    if (m >= M) continue;
                    const int wp = m / p.group, h = m - wp * p.group;
                    const long long row = row_of(p, w, b.i, wp);
                    if (row < 0) continue;
                    const uint16_t* src = p.q + row * p.q_stride + static_cast<size_t>(b.g * p.group + h) * D;
                    if constexpr (kPer == 4) {
                        const uint2 y = __ldg(reinterpret_cast<const uint2*>(src) + lane);
                        x[e][0] = y.x;
                        x[e][1] = y.y;
                    } else {
                        x[e][0] = __ldg(reinterpret_cast<const uint32_t*>(src) + lane);
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float f[kPer];
                    uint32_t top = 0;
#pragma unroll
                    for (int k = 0; k < kPer; ++k) {
                        f[k] = bf16_bits_to_float((x[e][k >> 1] >> (16 * (k & 1))) & 0xffffu);
                        f[k] = fmaf(f[k], 0.f, f[k]);            // an infinity becomes NaN
                        const uint32_t u = __float_as_uint(f[k]) & 0x7fffffffu;
                        if (u < 0x7f800000u) top = max(top, u);
                    }
                    top = __reduce_max_sync(0xffffffffu, top) >> 23;
                    // 2^(141 - top) puts the largest into [2^14, 2^15); it and its inverse
                    // stay normal (-113 at least, and 126)
                    const int shift = min(141 - static_cast<int>(top), 126);
                    const float mul = pow2f(shift);
                    uint32_t code[3] = {0, 0, 0};
#pragma unroll
                    for (int k = 0; k < kPer; k += 2) {
                        float a = f[k] * mul, c = f[k + 1] * mul;
#pragma unroll
                        for (int pl = 0; pl < 3; ++pl) {
                            const uint32_t two = f32x2_to_e5m2x2(a, c);
                            const float2 back = e5m2x2_to_f32x2(two);
                            a -= back.x;
                            c -= back.y;
                            code[pl] |= two << (8 * k);
                        }
                    }
                    const int r = r0 + e;
                    // bytes kPer * lane .. of row r, swizzled as TMA would have it
                    const int byte = kPer * lane, chunk = byte >> 4;
                    const int at = D == 128 ? r * 128 + ((chunk ^ (r & 7)) << 4) + (byte & 15)
                                            : r * 64 + ((chunk ^ ((r >> 1) & 3)) << 4) + (byte & 15);
#pragma unroll
                    for (int pl = 0; pl < 3; ++pl) {
                        if constexpr (kPer == 4) *reinterpret_cast<uint32_t*>(slot + pl * C::kPlane + at) = code[pl];
                        else *reinterpret_cast<uint16_t*>(slot + pl * C::kPlane + at) = static_cast<uint16_t>(code[pl]);
                    }
                    if (lane == 0) scale[r] = pow2f(-shift);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
        };
        // tile q by TMA: boxes of `box` whole tokens
        auto fetch = [&](const Blk& b, int q, uint8_t* slot, uint64_t* full) {
            if (lane == 0) {
                mbar_arrive_expect_tx(full, static_cast<uint32_t>(p.box) * p.group * D * 2);
#pragma unroll
                for (int h = 0; h < D / 64; ++h)
                    tma_load_3d(slot + h * (kTile * 128), &tmQ, full, h * 64, b.g * p.group, b.row0 + q * tokens);
            }
            __syncwarp();
            ++sent;
        };
        while (take(ok, b)) {
            if (!(b.flags & U_HAS)) continue;
            if constexpr (SMALL) {
                if (!(b.flags & U_NEWQ)) continue;
                float z[4];
                if (!rows_warp) lse_of(b, 0, z);
                ok = wait_or_fail(p, &bar.q_empty[qr.at], qr.empty());
                if (!ok) break;
                uint8_t* slot = smem + C::kQ + qr.at * C::kQBytes;
                if (!rows_warp) put_lse(b, 0, z, l2 + qr.at * kTile, bar.live[qr.at]);
                if constexpr (kPlanes) split(b, slot, cf + qr.at * kTile);
                else if (rows_warp && p.path) gather(b, 0, slot);
                if (!kPlanes && rows_warp && !p.path) {
                    fetch(b, 0, slot, &bar.q_full[qr.at]);
                } else {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.q_full[qr.at]);
                }
                qr.step();
            } else if (!rows_warp) {
                // a tile's are loaded two tiles before their place is free; without
                // a path the lane's columns only step from tile to tile (looked up
                // anew in each, a tile took this warp 1600 clocks)
                const float* at[4];
                int left[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const bool in = col_wp[k] < tokens;
                    left[k] = in ? b.M / p.group - b.q0 * tokens - col_wp[k] : 0;
                    at[k] = p.lse + (b.row0 + static_cast<long long>(b.q0) * tokens + (in ? col_wp[k] : 0)) * p.H +
                            b.g * p.group + col_h[k];
                }
                const int64_t step = static_cast<int64_t>(tokens) * p.H;
                auto load = [&](int q, float (&z)[4]) {
                    if (p.path) {
                        lse_of(b, q, z);
                        return;
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        z[k] = -INFINITY;
                        if (left[k] > 0) z[k] = __ldg(at[k]);
                        at[k] += step;
                        left[k] -= tokens;
                    }
                };
                auto put = [&](int q, const float (&z)[4]) {
                    ok = wait_or_fail(p, &bar.l_empty[lr.at], lr.empty());
                    if (!ok) return;
                    put_lse(b, q, z, l2 + lr.at * kTile, bar.live[lr.at]);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.l_full[lr.at]);
                    lr.step();
                };
                float z[2][4];
                load(b.q0, z[0]);
                for (int q = b.q0; q < b.q1 && ok; q += 2) {
                    if (q + 1 < b.q1) load(q + 1, z[1]);
                    put(q, z[0]);
                    if (!ok || q + 1 >= b.q1) break;
                    if (q + 2 < b.q1) load(q + 2, z[0]);
                    put(q + 1, z[1]);
                }
            } else {
                for (int q = b.q0; q < b.q1 && ok; ++q) {
                    ok = wait_or_fail(p, &bar.q_empty[qr.at], qr.empty());
                    if (!ok) break;
                    uint8_t* slot = smem + C::kQ + qr.at * C::kQBytes;
                    if (p.path) {
                        gather(b, q, slot);
                        if (lane == 0) mbar_arrive(&bar.q_full[qr.at]);
                    } else {
                        fetch(b, q, slot, &bar.q_full[qr.at]);
                    }
                    qr.step();
                }
            }
            if (!ok) break;
        }
        if (!ok && sent > 0)   // copies in flight land before the CTA may exit
            for (int k = 0; k < C::kQSlots; ++k)
                if (qr.turn > 0 || k < qr.at) mbar_wait(&bar.q_full[k], k < qr.at ? qr.turn & 1 : (qr.turn & 1) ^ 1);
    } else {
        // ------------------------------------------------------------------
        // weights: a thread per key
        // ------------------------------------------------------------------
        const int wg = (warp >> 2) & 1, half = warp >> 3;   // tile of keys; which tiles of rows, unless SMALL
        bool ok = true;
        uint32_t n_q = 0, n_mine = 0;     // tiles of rows; units with keys of this warpgroup
        uint32_t s_phase = 0;             // of the warpgroup's barrier of each S buffer
        Ring<2> jr;
        Ring<C::kS> sr;
        Ring<C::kQSlots> qr;
        Ring<C::kLStages> lr;
        Ring<kExpStages> xr;
        bool any_q = false;
        const float c0 = p.scale * kLog2e;
        bool big = false;                 // planes: a row's scale is above 1 (its elements from 2^15 on)
        Blk b;
        while (take(ok, b)) {
            if (SMALL && !(b.flags & U_HAS)) {
                // nothing to add: the old weights, or zeros (88 contexts of 40140, a window
                // of 314, 16 heads: 192 us; 896 when each unit was handed out alone)
                // (keys are counted from k0: a step from one near the largest length would pass 32 bits)
                const size_t at = (static_cast<size_t>(b.i) * p.c.heads + b.g) * p.stride + b.k0;
                const int keys = min(b.n - b.k0, b.q1 * kUnit), old_keys = b.ctx - b.k0;
                for (int key0 = tid; key0 < keys; key0 += 8 * kUnit) {
                    float x[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int key = key0 + k * kUnit;
                        x[k] = p.mass && key < keys && key < old_keys ? __ldcg(p.mass + at + key) : 0.f;
                    }
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (key0 + k * kUnit < keys) p.mass_out[at + key0 + k * kUnit] = x[k];
                }
                continue;
            }
            const int key = b.k0 + wg * kTile + (tid & 127);
            const bool mine = wg < b.tiles, held = mine && key < b.n;
            const bool has = b.flags & U_HAS;
            const size_t o = (static_cast<size_t>(b.i) * p.c.heads + b.g) * p.stride + key;
            float old = 0.f;
            if (held && p.mass && key < b.ctx && (b.flags & U_FIRST) && (b.flags & U_LAST)) old = __ldcg(p.mass + o);
            float sum = 0.f, lost = 0.f;
            if (has) {
                if (SMALL && (b.flags & U_NEWQ)) {
                    if (any_q) {
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bar.q_empty[qr.at]);
                        qr.step();
                    }
                    any_q = true;
                    ok = wait_or_fail(p, &bar.q_full[qr.at], qr.full());   // its -lse
                    if (!ok) break;
                    if constexpr (kPlanes) {
                        big = false;
                        for (int m = lane; m < b.M; m += 32) big = big || cf[qr.at * kTile + m] > 1.f;
                        big = __any_sync(0xffffffffu, big);
                    }
                }
                float c = c0;
                if constexpr (kPlanes) {
                    // this tile's exponents; the other warpgroup has the other's
                    if (mine) {
                        if (wg == 1) xr.step();
                        ok = wait_or_fail(p, &bar.x_full[xr.at], xr.full());
                        if (!ok) break;
                        c *= scale_of(smem[C::kExps + xr.at * kTile + (tid & 127)]);
                        xr.step();
                        if (wg == 0 && b.tiles == 2) xr.step();
                    } else {
                        xr.step();
                    }
                }
                if constexpr (E4M3 && !SMALL) {
                    // the tile's codes as bf16 into tensor memory, a key a thread, once
                    // the products of its last unit are complete: those of the last tile
                    // of rows may be the other half's. No phase of k_idle is missed: the
                    // next one's products wait for all these warps
                    if (mine && half < D / 64) {   // a half of the row each
                        uint4 x[4];
                        float s = 1.f;
#pragma unroll
                        for (int k = 0; k < 4; ++k) x[k] = make_uint4(0, 0, 0, 0);
                        if (held) {
                            int pg = page_of(p.c, b.i, key);
                            if (pg < 0) {
                                set_status(p.dev_status, SDM_DEV_BAD_PAGE);
                                pg = 0;
                            }
                            const size_t at = pool_row(p.c, pg, key) + (static_cast<size_t>(b.g) << p.c.page_shift);
                            const uint4* src = reinterpret_cast<const uint4*>(p.c.k + at * D + half * 64);
                            s = scale_of(__ldg(p.c.k_exp + at));
#pragma unroll
                            for (int k = 0; k < 4; ++k) x[k] = __ldg(src + k);
                        }
                        if (n_mine > 0) ok = wait_or_fail(p, &bar.k_idle[wg], (n_mine - 1) & 1);
                        if (!ok) break;
                        ++n_mine;
                        tc_fence_after();
                        uint32_t z[32];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t y[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const float2 f = f16x2_to_f32x2(e4m3x2_to_f16x2(static_cast<uint16_t>(y[e >> 1] >> (16 * (e & 1)))));
                                z[8 * k + e] = f32x2_to_bf16x2(f.x * s, f.y * s);
                            }
                        }
                        tmem_st32(tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + kTmemK + wg * (D / 2) + half * 32, z);
                        tmem_st_wait();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bar.kt_full[wg]);
                    }
                }
                // tiles q_lo .. q_hi - 1 of the rows see all of the warp's keys
                int q_lo = 0, q_hi = 0x7fffffff;
                {
                    const int key0 = b.k0 + wg * kTile + (warp & 3) * 32, key1 = key0 + 31;
                    if (key1 > b.ctx) q_lo = ((key1 - b.ctx) * p.group + p.sub - 1) / p.sub;
                    if (p.window > 0 && key1 >= p.sinks) {
                        const long long end = (static_cast<long long>(key0) - b.ctx + p.window) * p.group;
                        if (end < b.M) q_hi = end <= 0 ? 0 : static_cast<int>(end / p.sub);
                    }
                }
                for (int q = b.q0; q < b.q1 && ok; ++q) {
                    const float* lq = l2 + (SMALL ? qr.at : lr.at) * kTile;
                    // the halves take the tiles of rows in turn: one waits and loads
                    // while the other sums (8192 tokens, 32 / 8 heads: 222 us; 242 with
                    // half of every tile's columns each; 254 with six buffers of 64
                    // columns, whose products take as long as those of 128; 257 with
                    // 16 columns loaded while 16 are summed)
                    const bool turn = SMALL || static_cast<int>(n_q & 1) == half;
                    ++n_q;
                    if (!SMALL && turn) {
                        ok = wait_or_fail(p, &bar.l_full[lr.at], lr.full());
                        if (!ok) break;
                    }
                    if (wg == 1) sr.step();           // the other warpgroup's
                    if (mine && !turn) {
                        sr.step();
                        if (wg == 0 && b.tiles == 2) sr.step();
                    } else if (mine) {
                        const int cols = SMALL ? b.M : p.sub, first = q * p.sub;
                        // columns [lo, hi) see this key
                        int lo = 0, hi = min(cols, b.M - first);
                        const uint32_t* live = bar.live[SMALL ? qr.at : lr.at];
                        const bool some = q < q_lo || q >= q_hi || live[4];
                        if (some) {
                            if (key > b.ctx) lo = (key - b.ctx) * p.group - first;
                            if (p.window > 0 && key >= p.sinks) {
                                const long long end = static_cast<long long>(key) - b.ctx + p.window;   // rows below it see the key
                                if (end * p.group < b.M) hi = min(hi, static_cast<int>(max(end, 0ll)) * p.group - first);
                            }
                        }
                        ok = wait_or_fail(p, &bar.s_full[sr.at][SMALL ? wg : wg + 2 * half], (s_phase >> sr.at) & 1);
                        s_phase ^= 1u << sr.at;
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t s_at = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + sr.at * 128;
                        float2 acc[4] = {};
                        const float4* lp = reinterpret_cast<const float4*>(lq);
                        const float4* fp = reinterpret_cast<const float4*>(cf + qr.at * kTile);
                        auto add = [&](auto& x, int at) {   // columns from `at`
                            // columns behind a full tile's rows (65 at least) are products
                            // with zeros: NaN where the key has an infinity, and then the
                            // last of these 32 is (hidden in every such tile: 3 % of a prompt
                            // of 28 heads on 4)
                            const float end = __uint_as_float(x[sizeof(x) / 4 - 1]);
                            if (some || (at >= 64 && end != end)) hide(x, lo - at, hi - at, live[at / 32]);
                            add_weights<kPlanes, false>(x, c, lp + at / 4, fp + at / 4, acc);
                        };
                        if constexpr (SMALL) {
                            // few rows, or 32 columns loaded while the 32 before them
                            // are summed (two contexts of 150001 to 199999 with 7 rows
                            // a head: 48.3 us, 51.7 with 32 columns)
                            const int N = (cols + 31) & ~31;
                            if (kPlanes && big) {
                                acc[0].x = add_big(s_at, cols, lo, hi, live, c, lp, fp);
                            } else if (cols <= 16) {
                                uint32_t x[16];
                                tmem_ld16(s_at, x);
                                tmem_ld_wait();
                                add(x, 0);
                            } else {
                                uint32_t x[2][32];
                                tmem_ld32(s_at, x[0]);
#pragma unroll 1
                                for (int c1 = 0; c1 < N; c1 += 64) {
                                    tmem_ld_wait();
                                    if (c1 + 32 < N) tmem_ld32(s_at + c1 + 32, x[1]);
                                    add(x[0], c1);
                                    if (c1 + 32 >= N) break;
                                    tmem_ld_wait();
                                    if (c1 + 64 < N) tmem_ld32(s_at + c1 + 64, x[0]);
                                    add(x[1], c1 + 32);
                                }
                            }
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&bar.s_empty[sr.at]);
                        } else {
                            uint32_t x[32];
                            tmem_ld32(s_at, x);
                            tmem_ld_wait();
                            add(x, 0);
                            tmem_ld32(s_at + 32, x);
                            tmem_ld_wait();
                            add(x, 32);
                            tmem_ld32(s_at + 64, x);
                            tmem_ld_wait();
                            add(x, 64);
                            tmem_ld32(s_at + 96, x);
                            tmem_ld_wait();
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&bar.s_empty[sr.at]);
                            add(x, 96);
                        }
                        sr.step();
                        if (wg == 0 && b.tiles == 2) sr.step();
                        // the tiles' sums with what each addition loses: a key of a long
                        // prompt is the sum of thousands of weights
                        const float2 half = add2(add2(acc[0], acc[1]), add2(acc[2], acc[3]));
                        const float one = half.x + half.y - lost;
                        const float to = sum + one;
                        lost = to < INFINITY ? (to - sum) - one : 0.f;   // infinity loses nothing
                        sum = to;
                    }
                    if (!SMALL) {
                        __syncwarp();
                        if (turn && lane == 0) mbar_arrive(&bar.l_empty[lr.at]);
                        lr.step();
                    }
                }
                if (!ok) break;
            }
            if constexpr (!SMALL) {
                // the two halves' tiles of rows
                float* xch = reinterpret_cast<float*>(smem + C::kXch) + jr.at * kUnit + wg * kTile + (tid & 127);
                if (half == 1) {
                    ok = wait_or_fail(p, &bar.j_empty[wg][jr.at], jr.empty());
                    if (!ok) break;
                    *xch = sum;
                } else {
                    ok = wait_or_fail(p, &bar.j_full[wg][jr.at], jr.full());
                    if (!ok) break;
                    sum += *xch;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(half == 1 ? &bar.j_full[wg][jr.at] : &bar.j_empty[wg][jr.at]);
                jr.step();
                if (half == 1) continue;
            }
            if (held) {
                if ((b.flags & U_FIRST) && (b.flags & U_LAST)) p.mass_out[o] = old + sum;
                else ws.sum[(static_cast<size_t>(blockIdx.x) * 2 + ((b.flags & U_FIRST) ? 1 : 0)) * kUnit + wg * kTile + (tid & 127)] = sum;
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kSoft + 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// Adds the parts of the unit that a share starts and does not finish, in order.
__global__ void __launch_bounds__(kUnit) weigh_join_kernel(const WeighParams p, const Scratch ws, int grid) {
    pdl_wait();
    pdl_trigger();
    const int c = blockIdx.x;
    const Part s = ws.part[c];
    if (!s.rest) return;
    const int key = s.k0 + threadIdx.x;
    const float* sums = ws.sum + threadIdx.x;
    float sum = sums[(2 * static_cast<size_t>(c) + 1) * kUnit];
    for (int k = c + 1; k < grid; ++k) {
        const int head = ws.part[k].head;
        if (head) sum += sums[2 * static_cast<size_t>(k) * kUnit];
        if (head == 1) break;
    }
    if (key >= s.n) return;
    const size_t o = (static_cast<size_t>(s.i) * p.c.heads + s.g) * p.stride + key;
    p.mass_out[o] = (key < s.ctx && p.mass ? __ldcg(p.mass + o) : 0.f) + sum;
}

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
                            cudaSuccess && q == cudaDriverEntryPointSuccess;
        return ok ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f) : nullptr;
    }();
    return fn;
}

bool encode_q(CUtensorMap* map, const WeighParams& p) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(p.c.D), static_cast<cuuint64_t>(p.H), static_cast<cuuint64_t>(p.rows)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(p.c.D) * 2, static_cast<cuuint64_t>(p.q_stride) * 2};
    cuuint32_t box[3] = {64u, static_cast<cuuint32_t>(p.group), static_cast<cuuint32_t>(p.box)};
    cuuint32_t el[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(p.q), dims, strides, box, el,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// rows = (page, head, slot); a box is one page of one head, 128 bytes (e4m3 with 64-wide heads: 64) across
bool encode_k(CUtensorMap* map, const CacheView& c) {
    auto fn = encode_fn();
    if (!fn) return false;
    const int es = c.e4m3 ? 1 : 2, cols = c.e4m3 ? c.D : 64;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(c.D), static_cast<cuuint64_t>(c.n_pages) * c.heads << c.page_shift};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(c.D) * es};
    cuuint32_t box[2] = {static_cast<cuuint32_t>(cols), 1u << c.page_shift};
    cuuint32_t el[2] = {1, 1};
    return fn(map, c.e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, c.k, dims, strides, box,
              el, CU_TENSOR_MAP_INTERLEAVE_NONE, cols * es == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool E4M3, bool SMALL>
cudaError_t launch_one(const WeighParams& p, void* work, cudaStream_t s) {
    using C = Cfg<D, E4M3, SMALL>;
    constexpr int kTotal = C::kBars + static_cast<int>(sizeof(Bars<C::kKSlots, C::kQSlots, C::kLStages, C::kRing, C::kS>));
    static_assert(kTotal <= 232448, "shared memory");
    static SmemLimit limit;
    const cudaError_t raised = limit.raise(weigh_kernel<D, E4M3, SMALL>, kTotal);
    if (raised != cudaSuccess) return raised;
    CUtensorMap tmK;
    if (!encode_k(&tmK, p.c)) return cudaErrorInvalidValue;
    CUtensorMap tmQ = tmK;
    if (!C::kPlanes && p.rows > 0 && !encode_q(&tmQ, p)) return cudaErrorInvalidValue;
    const int grid = num_sms();
    Scratch ws = {};
    if (!SMALL) {
        ws.part = static_cast<Part*>(work);
        ws.sum = reinterpret_cast<float*>(static_cast<uint8_t*>(work) + align256(sizeof(Part) * grid));
    }
    const cudaError_t e = launch_pdl(weigh_kernel<D, E4M3, SMALL>, dim3(grid), dim3(C::kThreads), kTotal, s, tmK, tmQ, p, ws);
    if (e != cudaSuccess || SMALL) return e;
    return launch_pdl(weigh_join_kernel, dim3(grid), dim3(kUnit), 0, s, p, ws, grid);
}

// Query rows of a tile: those of as many whole tokens as it holds.
inline int tile_rows(int group) { return kTile / group * group; }

template <int D, bool E4M3>
cudaError_t launch_form(const WeighParams& p, void* ws, cudaStream_t s) {
    const bool small = static_cast<long long>(p.max_count) * p.group <= p.sub;
    return small ? launch_one<D, E4M3, true>(p, ws, s) : launch_one<D, E4M3, false>(p, ws, s);
}

}  // namespace

size_t weigh_workspace(int max_count, int H, int kv_heads) {
    if (max_count <= 0 || H <= 0 || kv_heads <= 0 || H / kv_heads > kTile || H < kv_heads) return 0;
    const int group = H / kv_heads;
    if (static_cast<long long>(max_count) * group <= tile_rows(group)) return 0;
    const size_t grid = num_sms();
    return align256(sizeof(Part) * grid) + grid * 2 * kUnit * sizeof(float);
}

cudaError_t launch_weigh(const WeighParams& p, void* ws, cudaStream_t s) {
    WeighParams q = p;
    q.sub = tile_rows(p.group);
    q.box = std::max(1, std::min(p.max_count, q.sub / p.group));
    if (p.c.D == 128) return p.c.e4m3 ? launch_form<128, true>(q, ws, s) : launch_form<128, false>(q, ws, s);
    return p.c.e4m3 ? launch_form<64, true>(q, ws, s) : launch_form<64, false>(q, ws, s);
}

}  // namespace sdm
