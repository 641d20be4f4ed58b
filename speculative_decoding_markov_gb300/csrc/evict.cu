// evict.cu - a paged cache cut to `keep` tokens per request and kv head: the
// first positions, the last ones, then those of largest attention weight.
//
// A cluster of CTAs per (request, kv head), each with an equal run of slots.
//   1. Slots become 32-bit keys in order of their weight; a first or last
//      position's is the largest.  The keep-th largest key is found by its
//      digits, the first of 11 bits, which tells weights of a few octaves apart:
//      a histogram each, summed over the cluster.
//   2. Slots above that key are kept, and of its equals the lowest, by counts
//      in slot order.  Kept tokens that lie in front of slot `keep` stay where
//      they are; the j-th of the others moves into the j-th slot that becomes
//      free there (keys hold their rotation, so their order in the cache is of
//      no account).  Sources lie behind `keep`, destinations before it, so
//      moves need no order.
// Only what has to move is moved: of a cache that runs full by 8 tokens a
// cycle, 8 rows, not the 2048 that kept their place.
//
// What bounds it: 64 such caches of 8 heads x 128 (11.9 us) a chain of look-ups
// and barriers; five prompts of up to 30000 tokens cut to 4096 (28 heads on 4,
// e4m3, 35 us) the barriers of clusters of 8 and the moves' scattered rows.
#include <cooperative_groups.h>

#include <algorithm>

#include "paged.cuh"

namespace sdm {
namespace {

namespace cg = cooperative_groups;

constexpr int kBins = 2048;
constexpr int kMoves = 4;          // moves of a thread in flight together
constexpr int kList = 1024;        // keys that share the first digits
constexpr int kMost = 48 * 1024;   // keys a CTA can hold
constexpr int kFew = 16;           // slots to go that are looked for one by one

// Of a run of slots: those above the keep-th largest key and equal to it, in
// front of slot `keep` and behind.
struct Counts {
    int above_lo, equal_lo, above_hi, equal_hi;
};

template <int THREADS>
struct Shared {
    int hist[kBins];       // this CTA's
    int all[kBins];        // the cluster's, in its first CTA
    int sum[THREADS / 32];
    Counts warp[THREADS / 32];
    Counts mine;
    int pick, before, last, listed;
    uint32_t list[kList];
    unsigned long long least[2][THREADS / 32];
    int gone[kFew], src[kFew], dst[kFew];
};

struct Held {              // a request's slots
    int n, ctx;            // held before the cut; numbered by pos
    long long start, end;  // position of slot ctx, and one past the last
    int bad;
};

__device__ __forceinline__ Held held_of(const EvictParams& p, int i) {
    Held h;
    h.bad = 0;
    const long long most = min(min(table_tokens(p.c), static_cast<long long>(p.stride)), 0x7fffffffll);
    int ctx = __ldg(p.ctx + i), more = p.count ? __ldg(p.count + i) : 0;
    if (ctx < 0 || more < 0) h.bad = SDM_DEV_BAD_WINDOW;
    ctx = max(ctx, 0);
    more = max(more, 0);
    h.start = p.start ? __ldg(p.start + i) : ctx;
    h.end = h.start + more;
    if (static_cast<long long>(ctx) + more > most) {
        h.bad |= SDM_DEV_BAD_PAGE;
        ctx = static_cast<int>(min(static_cast<long long>(ctx), most));
        more = static_cast<int>(min(static_cast<long long>(more), most - ctx));
    }
    h.ctx = ctx;
    h.n = ctx + more;
    return h;
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) evict_kernel(const EvictParams p) {
    constexpr int kWarps = kThreads / 32;
    __shared__ Shared<kThreads> sh;
    extern __shared__ uint32_t keys[];
    pdl_wait();
    pdl_trigger();
    cg::cluster_group cluster = cg::this_cluster();
    const int C = cluster.num_blocks(), rank = cluster.block_rank();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tid = threadIdx.x;
    const int item = blockIdx.x / C, i = item / p.c.heads, g = item % p.c.heads;
    const Held h = held_of(p, i);
    const int keep = p.keep;
    if (rank == 0 && g == 0 && tid == 0) {
        if (h.bad) set_status(p.dev_status, h.bad);
        p.length[i] = min(h.n, keep);
        if (p.next) p.next[i] = static_cast<int32_t>(h.end);
    }
    const size_t base = static_cast<size_t>(item) * p.stride;
    const float* mass = p.mass + base;
    const int32_t* pos = p.pos + base;
    float* mass_out = p.mass_out + base;
    int32_t* pos_out = p.pos_out + base;
    auto where = [&](int s) {
        return s < h.ctx ? __ldcg(pos + s) : static_cast<int32_t>(h.start + (s - h.ctx));
    };
    // the CTA's slots, whole warps' worth
    const int per = (((h.n + C - 1) / C) + 31) & ~31;
    const int s0 = static_cast<int>(min(static_cast<long long>(per) * rank, static_cast<long long>(h.n)));
    const int s1 = static_cast<int>(min(static_cast<long long>(s0) + per, static_cast<long long>(h.n)));
    const int run = s1 - s0;   // slots are counted from s0: near the largest length a step from one would pass 32 bits
    const bool same = mass_out == mass && pos_out == pos, cut = h.n > keep;
    auto key = [&](int32_t at, float m) {
        if (at < p.sinks || at >= h.end - p.recent) return 0xffffffffu;
        return m == m ? min(ordered_bits(m), 0xfffffffeu) : 0u;
    };
    // The keys stay in shared memory; a run of slots that does not fit is
    // looked up again wherever its keys are wanted.
    const bool fits = per <= p.room;
    const bool few = cut && C == 1 && fits && h.n - keep <= kFew;
    if (cut && !few) {
        for (int b = tid; b < kBins; b += kThreads) {
            sh.hist[b] = 0;
            sh.all[b] = 0;
        }
        if (tid == 0) sh.listed = 0;
        __syncthreads();
    }
    for (int b = 0; b < run; b += 4 * kThreads) {
        int32_t at[4];
        float m[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = b + j * kThreads + tid;
            if (r < run) {
                at[j] = where(s0 + r);
                m[j] = __ldcg(mass + s0 + r);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = b + j * kThreads + tid;
            if (r >= run) continue;
            const int s = s0 + r;
            if (cut) {
                const uint32_t k = key(at[j], m[j]);
                if (fits) keys[r] = k;
                if (!few) atomicAdd(&sh.hist[k >> 21], 1);
            }
            if (s < keep && !(same && s < h.ctx)) {   // those that stay; the others' places are overwritten below
                mass_out[s] = m[j];
                pos_out[s] = at[j];
            }
        }
    }
    if (!cut) return;   // the whole cluster
    auto key_of = [&](int s) { return fits ? keys[s - s0] : key(where(s), __ldcg(mass + s)); };
    int total = 0;         // moves
    int32_t* from = p.moves + 2 * static_cast<size_t>(item) * p.most;
    int32_t* to = from + p.most;
    if (few) {
        // A full cache that has grown by a few tokens (every cycle of decoding):
        // the slots that go, one by one: the least key, among equals the last
        // slot.  64 caches of 2048 and up to 8: 11.4 us, by digits 17.9.
        const int e = h.n - keep;
        auto mark = [&](int s) { return (static_cast<unsigned long long>(keys[s]) << 32) | static_cast<uint32_t>(~s); };
        unsigned long long best = ~0ull;
        for (int s = tid; s < h.n; s += kThreads) best = min(best, mark(s));   // of the keys this thread wrote
        for (int r = 0; r < e; ++r) {
            const uint32_t hi = __reduce_min_sync(0xffffffffu, static_cast<uint32_t>(best >> 32));
            const uint32_t low =
                __reduce_min_sync(0xffffffffu, (best >> 32) == hi ? static_cast<uint32_t>(best) : 0xffffffffu);
            if (lane == 0) sh.least[r & 1][warp] = (static_cast<unsigned long long>(hi) << 32) | low;
            __syncthreads();
            unsigned long long least = sh.least[r & 1][0];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) least = min(least, sh.least[r & 1][w]);
            const int s = static_cast<int>(~static_cast<uint32_t>(least));
            if (tid == 0) sh.gone[r] = s;
            if (best == least) {
                best = ~0ull;
                for (int t = tid; t < h.n; t += kThreads) {
                    const unsigned long long x = mark(t);
                    if (x > least) best = min(best, x);
                }
            }
        }
        __syncthreads();
        if (warp == 0) {
            const int s = lane < e ? sh.gone[lane] : 0x7fffffff;
            int before = 0;
            bool stays = true;      // slot keep + lane
            for (int r = 0; r < e; ++r) {
                const int o = __shfl_sync(0xffffffffu, s, r);
                before += o < s;
                stays = stays && o != keep + lane;
            }
            const unsigned moves = __ballot_sync(0xffffffffu, lane < e && stays);
            if (s < keep) sh.dst[before] = s;
            if ((moves >> lane) & 1u) sh.src[__popc(moves & ((1u << lane) - 1))] = keep + lane;
            if (lane == 0) sh.before = __popc(moves);
        }
        __syncthreads();
        total = sh.before;
    } else {
        // 1. the keep-th largest key, digit by digit: `need` of the keys that share
        // the digits found are wanted
        uint32_t found = 0, mask = 0;
        int need = keep;
        Shared<kThreads>* first = C > 1 ? cluster.map_shared_rank(&sh, 0) : &sh;
        auto meet = [&]() {
            if (C > 1) cluster.sync();
            else __syncthreads();
        };
        // 11 bits, then 7 at a time by one warp, or in clusters, whose every digit
        // costs three of their barriers, 11 and 10
#pragma unroll 1
        for (int d = 0, shift = 21; ; ++d) {
            const int width = d == 0 ? 11 : C == 1 ? 7 : min(shift, 11);
            if (d > 0) shift -= width;
            const int bins = 1 << width;
            if (d > 0) {   // the first digit's were counted as the keys were made
                for (int b = tid; b < bins; b += kThreads) {
                    sh.hist[b] = 0;
                    if (C > 1 && rank == 0) sh.all[b] = 0;
                }
                if (C > 1) cluster.sync();   // the first CTA's counts are clear
                else __syncthreads();
                const int listed = d > 1 ? sh.listed : kList + 1;
                if (listed <= kList) {
                    for (int s = tid; s < listed; s += kThreads)
                        if ((sh.list[s] & mask) == found) atomicAdd(&sh.hist[(sh.list[s] >> shift) & (bins - 1)], 1);
                } else {
#pragma unroll 4
                    for (int r = tid; r < run; r += kThreads) {
                        const uint32_t k = key_of(s0 + r);
                        if ((k & mask) != found) continue;
                        atomicAdd(&sh.hist[(k >> shift) & (bins - 1)], 1);
                        if (d == 1) {
                            const int at = atomicAdd(&sh.listed, 1);
                            if (at < kList) sh.list[at] = k;
                        }
                    }
                }
            }
            __syncthreads();
            // the bins that have any to the first CTA (each CTA reading all of the
            // others' bins took 33000 clocks a digit in clusters of 8)
            if (C > 1) {
                if (d == 0) cluster.sync();   // the first CTA's counts are clear
                for (int b = tid; b < bins; b += kThreads)
                    if (const int n = sh.hist[b]) atomicAdd(&first->all[b], n);
                cluster.sync();
            }
            // the bin of the need-th key from the top
            const int* hist = C > 1 ? sh.all : sh.hist;
            const bool wide = bins > 128;
            if (rank == 0 && (wide || warp == 0)) {
                constexpr int kPer = kBins / kThreads;   // bins a thread; 4 a lane of one warp for the short digits
                const int per_bins = wide ? bins / kThreads : 4;
                const int b0 = bins - per_bins - per_bins * tid;
                int n[kPer], all = 0;
#pragma unroll
                for (int j = 0; j < kPer; ++j) {
                    n[j] = j < per_bins ? hist[b0 + per_bins - 1 - j] : 0;
                    all += n[j];
                }
                int incl = all;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += y;
                }
                int before = incl - all;
                if (wide) {
                    if (lane == 31) sh.sum[warp] = incl;
                    __syncthreads();
                    for (int w = 0; w < warp; ++w) before += sh.sum[w];
                }
#pragma unroll
                for (int j = 0; j < kPer; ++j) {
                    if (before < need && need <= before + n[j]) {
                        sh.pick = b0 + per_bins - 1 - j;
                        sh.before = before;
                        sh.last = need == before + n[j];   // all of the bin
                    }
                    before += n[j];
                }
            }
            meet();
            found |= static_cast<uint32_t>(first->pick) << shift;
            mask |= static_cast<uint32_t>(bins - 1) << shift;
            need -= first->before;
            if (first->last && shift > 0) {
                // every key with these digits is wanted, so the lower ones need not
                // be found.  (Not all are 0: fewer than all keys are wanted.)
                found -= 1;
                need = 0;
                break;
            }
            if (shift == 0) break;
            meet();   // before the picks are overwritten
        }
        // 2. which slots are kept: above `found`, and the first `need` of its equals.
        // A warp takes neighbouring groups of 32 slots, and a lane then one group of
        // 32 that it has looked at: few instructions a slot bound this kernel.
        const int groups = (run + 31) / 32, each = (groups + kWarps - 1) / kWarps;
        const int w0 = min(groups, warp * each), w1 = min(groups, w0 + each);
        // lane k: which slots of group k0 + k are above and equal, and which lie in front of `keep`
        auto look = [&](int k0, unsigned& above, unsigned& equal, unsigned& valid, unsigned& lo) {
            above = equal = 0;
            const int n = min(32, w1 - k0);
#pragma unroll 4
            for (int k = 0; k < n; ++k) {
                const int s = s0 + (k0 + k) * 32 + lane;
                const uint32_t x = s < s1 ? key_of(s) : 0u;
                const unsigned a = __ballot_sync(0xffffffffu, s < s1 && x > found);
                const unsigned e = __ballot_sync(0xffffffffu, s < s1 && x == found);
                if (lane == k) {
                    above = a;
                    equal = e;
                }
            }
            auto below = [](int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1; };
            const int s = s0 + min(k0 + lane, w1) * 32;
            valid = lane < n ? below(s1 - s) : 0u;
            lo = below(keep - s);
        };
        unsigned above, equal, valid, lo;
        Counts c = {};
        for (int k0 = w0; k0 < w1; k0 += 32) {
            look(k0, above, equal, valid, lo);
            c.above_lo += __popc(above & lo);
            c.equal_lo += __popc(equal & lo);
            c.above_hi += __popc(above & ~lo);
            c.equal_hi += __popc(equal & ~lo);
        }
        c.above_lo = __reduce_add_sync(0xffffffffu, c.above_lo);
        c.equal_lo = __reduce_add_sync(0xffffffffu, c.equal_lo);
        c.above_hi = __reduce_add_sync(0xffffffffu, c.above_hi);
        c.equal_hi = __reduce_add_sync(0xffffffffu, c.equal_hi);
        if (lane == 0) sh.warp[warp] = c;
        __syncthreads();
        if (C > 1 && tid == 0) {
            Counts t = {};
            for (int w = 0; w < kWarps; ++w) {
                t.above_lo += sh.warp[w].above_lo;
                t.equal_lo += sh.warp[w].equal_lo;
                t.above_hi += sh.warp[w].above_hi;
                t.equal_hi += sh.warp[w].equal_hi;
            }
            sh.mine = t;
        }
        if (C > 1) cluster.sync();
        // what stands before this warp's slots: equals, kept ones in front, movers.
        // Runs are in slot order, so a run's kept equals follow from the equals before it.
        int eq = 0, kept_lo = 0, mover = 0;
        {
            int all_eq = 0, all_kept = 0;
            auto pass = [&](const Counts& t, int& eq, int& kept, int& movers) {
                kept += t.above_lo + min(max(need - eq, 0), t.equal_lo);
                movers += t.above_hi + min(max(need - eq - t.equal_lo, 0), t.equal_hi);
                eq += t.equal_lo + t.equal_hi;
            };
            if (C > 1)
                for (int k = 0; k < C; ++k) {
                    const Counts t = *cluster.map_shared_rank(&sh.mine, k);
                    if (k < rank) pass(t, eq, kept_lo, mover);
                    pass(t, all_eq, all_kept, total);
                }
            for (int w = 0; w < kWarps; ++w) {
                if (w < warp) pass(sh.warp[w], eq, kept_lo, mover);
                if (C == 1) pass(sh.warp[w], all_eq, all_kept, total);
            }
        }
        int hole = min(s0 + w0 * 32, keep) - kept_lo;
        auto scan = [&](int n) {   // exclusive, over the warp
            int incl = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            return incl - n;
        };
        for (int k0 = w0; k0 < w1; k0 += 32) {
            if (w1 - w0 > 32) look(k0, above, equal, valid, lo);   // else as they are
            // the group's equals that are still wanted: its lowest ones
            const int eq_n = __popc(equal), eq_at = eq + scan(eq_n);
            unsigned kept_eq = equal;
            for (int k = max(need - eq_at, 0); k < __popc(kept_eq);) kept_eq &= ~(0x80000000u >> __clz(kept_eq));
            const unsigned kept = above | kept_eq;
            unsigned holes = valid & lo & ~kept, movers = kept & ~lo;
            int h_at = hole + scan(__popc(holes)), m_at = mover + scan(__popc(movers));
            eq += __reduce_add_sync(0xffffffffu, eq_n);
            hole += __reduce_add_sync(0xffffffffu, __popc(holes));
            mover += __reduce_add_sync(0xffffffffu, __popc(movers));
            const int s = s0 + min(k0 + lane, w1) * 32;
            // Keys that are looked up again are other ones if weights or positions
            // change meanwhile (which a call does not allow): no place is taken on trust.
            for (; holes; holes &= holes - 1, ++h_at)
                if (static_cast<unsigned>(h_at) < p.most) to[h_at] = s + __ffs(holes) - 1;
            for (; movers; movers &= movers - 1, ++m_at)
                if (static_cast<unsigned>(m_at) < p.most) from[m_at] = s + __ffs(movers) - 1;
        }
        total = static_cast<int>(min(static_cast<long long>(total), static_cast<long long>(p.most)));
        meet();   // the lists are whole
    }

    // 3. the moves, kMoves a thread together
    const int row_bytes = p.c.D * (p.c.e4m3 ? 1 : 2);
    const int pieces = row_bytes >> 4;                  // 16-byte pieces of a row: 4, 8 or 16
    const int per_move = 2 * pieces;
    const int lane_of = tid % per_move, slots = C * kThreads / per_move;
    const bool is_v = lane_of >= pieces;
    const int piece = lane_of % pieces;
    uint8_t* pool = is_v ? p.c.v : p.c.k;
    uint8_t* exps = is_v ? p.c.v_exp : p.c.k_exp;
    const size_t head = static_cast<size_t>(g) << p.c.page_shift;
    int bad = 0;
    for (int j0 = (rank * kThreads + tid) / per_move; j0 < total; j0 += kMoves * slots) {
        int src[kMoves], dst[kMoves];
        int32_t at[kMoves];
        float m[kMoves];
        uint4 x[kMoves];
        uint8_t e[kMoves];
        long long rd[kMoves];
#pragma unroll
        for (int q = 0; q < kMoves; ++q) {
            const int j = j0 + q * slots;
            src[q] = j >= total ? -1 : few ? sh.src[j] : __ldcg(from + j);
            dst[q] = j >= total ? -1 : few ? sh.dst[j] : __ldcg(to + j);
            if (src[q] >= h.n || static_cast<unsigned>(dst[q]) >= static_cast<unsigned>(keep)) src[q] = -1;
        }
#pragma unroll
        for (int q = 0; q < kMoves; ++q) {
            rd[q] = -1;
            if (src[q] < 0) continue;
            if (lane_of == 0) {
                m[q] = __ldcg(mass + src[q]);
                at[q] = where(src[q]);
            }
            const int pg_s = page_of(p.c, i, src[q]), pg_d = page_of(p.c, i, dst[q]);
            if (pg_s < 0 || pg_d < 0) {
                bad = SDM_DEV_BAD_PAGE;
                continue;
            }
            const size_t rs = pool_row(p.c, pg_s, src[q]) + head;
            rd[q] = static_cast<long long>(pool_row(p.c, pg_d, dst[q]) + head);
            x[q] = *reinterpret_cast<const uint4*>(pool + rs * row_bytes + piece * 16);
            if (p.c.e4m3 && piece == 0) e[q] = exps[rs];
        }
#pragma unroll
        for (int q = 0; q < kMoves; ++q) {
            if (src[q] < 0) continue;
            if (lane_of == 0) {
                mass_out[dst[q]] = m[q];
                pos_out[dst[q]] = at[q];
            }
            if (rd[q] < 0) continue;
            *reinterpret_cast<uint4*>(pool + rd[q] * row_bytes + piece * 16) = x[q];
            if (p.c.e4m3 && piece == 0) exps[rd[q]] = e[q];
        }
    }
    if (bad) set_status(p.dev_status, bad);
    if (C > 1) cluster.sync();   // nobody leaves while its counts are read
}

template <int THREADS>
cudaError_t launch_one(const EvictParams& p, int C, cudaStream_t s) {
    static SmemLimit limit;
    const cudaError_t raised = limit.raise(evict_kernel<THREADS>, kMost * 4);
    if (raised != cudaSuccess) return raised;
    EvictParams q = p;
    const long long per = ((p.stride + C - 1) / C + 31) / 32 * 32;
    q.room = static_cast<int>(std::min<long long>(per, kMost));
    return launch_cluster(evict_kernel<THREADS>, dim3(static_cast<unsigned>(static_cast<long long>(p.R) * p.c.heads * C)),
                          dim3(THREADS), C, q.room * 4, s, q);
}

}  // namespace

// The moves' sources and destinations: at most min(keep, stride - keep) a head.
static int64_t most_moves(int64_t stride, int keep) { return std::max<int64_t>(0, std::min<int64_t>(keep, stride - keep)); }

size_t evict_workspace(int R, int kv_heads, int64_t stride, int keep) {
    if (R <= 0 || kv_heads <= 0 || stride <= 0 || keep <= 0) return 0;
    return static_cast<size_t>(R) * kv_heads * most_moves(stride, keep) * 2 * sizeof(int32_t);
}

cudaError_t launch_evict(const EvictParams& p, cudaStream_t s) {
    EvictParams q = p;
    q.most = most_moves(p.stride, p.keep);
    const long long items = static_cast<long long>(p.R) * p.c.heads;
    int C = 1;
    // more CTAs a head while the SMs have room, or while its keys do not fit in one
    // (14 requests of up to 148331 tokens and 16 heads, cut to 314: 194 us; 700 in one CTA,
    // which looks its keys up anew)
    while (C < 8 && p.stride / (2 * C) >= 2048 && (items * C * 2 <= 2LL * num_sms() || p.stride / C > kMost)) C *= 2;
    // short runs: smaller CTAs, more of which are on an SM together
    return p.stride / C <= 4096 && C == 1 ? launch_one<256>(q, C, s) : launch_one<512>(q, C, s);
}

}  // namespace sdm
