// evict.cu - a paged cache cut to `keep` tokens per request and kv head: the
// first positions, the last ones, then those of largest attention weight.
//
// A cluster of CTAs per (request, kv head), each with an equal run of slots.
//   1. Slots become 32-bit keys in order of their weight; a first or last
//      position's is the largest.  The keep-th largest key is found by its
//      digits (11, 11 and 10 bits): a histogram each, summed over the cluster.
//   2. Slots above that key are kept, and of its equals the lowest, by counts
//      in slot order.  Kept tokens that lie in front of slot `keep` stay where
//      they are; the j-th of the others moves into the j-th slot that becomes
//      free there (keys hold their rotation, so their order in the cache is of
//      no account).  Sources lie behind `keep`, destinations before it, so
//      moves need no order.
// Only what has to move is moved: of a cache that runs full by 8 tokens a
// cycle, 8 rows, not the 2048 that kept their place.
#include <cooperative_groups.h>

#include <algorithm>

#include "paged.cuh"

namespace sdm {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;

struct Shared {
    int hist[kBins];
    int warp[kWarps][3];
    int mine[4];           // of this CTA: equals; then holes, movers
    int pick, before;
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

__global__ void __launch_bounds__(kThreads) evict_kernel(const EvictParams p) {
    __shared__ Shared sh;
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
    const bool same = mass_out == mass && pos_out == pos, cut = h.n > keep;
    auto key = [&](int32_t at, float m) {
        if (at < p.sinks || at >= h.end - p.recent) return 0xffffffffu;
        return m == m ? min(ordered_bits(m), 0xfffffffeu) : 0u;
    };
    // The keys stay in shared memory; a run of slots that does not fit is
    // looked up again wherever its keys are wanted.
    const bool fits = per <= p.room;
    for (int b = s0; b < s1; b += 4 * kThreads) {
        int32_t at[4];
        float m[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int s = b + j * kThreads + tid;
            if (s < s1) {
                at[j] = where(s);
                m[j] = __ldcg(mass + s);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int s = b + j * kThreads + tid;
            if (s >= s1) continue;
            if (cut && fits) keys[s - s0] = key(at[j], m[j]);
            if (s < keep && !(same && s < h.ctx)) {   // those that stay; the others' places are overwritten below
                mass_out[s] = m[j];
                pos_out[s] = at[j];
            }
        }
    }
    if (!cut) return;   // the whole cluster
    auto key_of = [&](int s) { return fits ? keys[s - s0] : key(where(s), __ldcg(mass + s)); };
    // 1. the keep-th largest key
    uint32_t found = 0, mask = 0;
    int need = keep;       // rank of the wanted key among those that share the digits found
#pragma unroll 1
    for (int d = 0; d < 3; ++d) {
        const int shift = d == 0 ? 21 : d == 1 ? 10 : 0;
        const uint32_t digits = d == 2 ? 1023u : 2047u;
        for (int b = tid; b < kBins; b += kThreads) sh.hist[b] = 0;
        __syncthreads();
        for (int s = s0 + tid; s < s1; s += kThreads) {
            const uint32_t k = key_of(s);
            if ((k & mask) == found) atomicAdd(&sh.hist[(k >> shift) & digits], 1);
        }
        if (C > 1) cluster.sync();
        else __syncthreads();
        // four bins a thread, from the top; their counts over the cluster
        int n4[4], all = 0;
        const int b0 = kBins - 4 - 4 * tid;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            n4[j] = 0;
            for (int k = 0; k < C; ++k) n4[j] += C > 1 ? cluster.map_shared_rank(sh.hist, k)[b0 + 3 - j] : sh.hist[b0 + 3 - j];
            all += n4[j];
        }
        int incl = all;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) sh.warp[warp][0] = incl;
        __syncthreads();
        int before = incl - all;
        for (int w = 0; w < warp; ++w) before += sh.warp[w][0];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (before < need && need <= before + n4[j]) {
                sh.pick = b0 + 3 - j;
                sh.before = before;
            }
            before += n4[j];
        }
        if (C > 1) cluster.sync();
        else __syncthreads();
        found |= static_cast<uint32_t>(sh.pick) << shift;
        mask |= digits << shift;
        need -= sh.before;
        __syncthreads();
    }
    // 2. which slots are kept: above `found`, and the first `need` of its equals
    // a warp takes neighbouring groups of 32 slots
    const int groups = (s1 - s0 + 31) / 32, each = (groups + kWarps - 1) / kWarps;
    const int w0 = min(groups, warp * each), w1 = min(groups, w0 + each);
    int equals = 0;
    for (int k = w0; k < w1; ++k) {
        const int s = s0 + k * 32 + lane;
        equals += __popc(__ballot_sync(0xffffffffu, s < s1 && key_of(s) == found));
    }
    if (lane == 0) sh.warp[warp][0] = equals;
    __syncthreads();
    if (tid == 0) {
        int sum = 0;
        for (int w = 0; w < kWarps; ++w) sum += sh.warp[w][0];
        sh.mine[0] = sum;
    }
    if (C > 1) cluster.sync();
    else __syncthreads();
    int eq = 0;
    for (int k = 0; k < rank; ++k) eq += cluster.map_shared_rank(sh.mine, k)[0];
    for (int w = 0; w < warp; ++w) eq += sh.warp[w][0];
    const int eq0 = eq;
    auto kept_of = [&](int s, int& eq) {   // by the whole warp, in order
        const uint32_t k = s < s1 ? key_of(s) : 0u;
        const bool even = s < s1 && k == found;
        const unsigned who = __ballot_sync(0xffffffffu, even);
        const bool r = s < s1 && (k > found || (even && eq + __popc(who & ((1u << lane) - 1)) < need));
        eq += __popc(who);
        return r;
    };
    int holes = 0, movers = 0;
    for (int k = w0; k < w1; ++k) {
        const int s = s0 + k * 32 + lane;
        const bool kept = kept_of(s, eq);
        holes += __popc(__ballot_sync(0xffffffffu, s < min(s1, keep) && !kept));
        movers += __popc(__ballot_sync(0xffffffffu, s >= keep && kept));
    }
    if (lane == 0) {
        sh.warp[warp][1] = holes;
        sh.warp[warp][2] = movers;
    }
    __syncthreads();
    if (tid == 0) {
        int a = 0, b = 0;
        for (int w = 0; w < kWarps; ++w) a += sh.warp[w][1], b += sh.warp[w][2];
        sh.mine[1] = a;
        sh.mine[2] = b;
    }
    if (C > 1) cluster.sync();
    else __syncthreads();
    int hole = 0, mover = 0, total = 0;
    for (int k = 0; k < C; ++k) {
        const int* o = C > 1 ? cluster.map_shared_rank(sh.mine, k) : sh.mine;
        if (k < rank) hole += o[1], mover += o[2];
        total += o[1];
    }
    for (int w = 0; w < warp; ++w) hole += sh.warp[w][1], mover += sh.warp[w][2];
    int32_t* from = p.moves + 2 * static_cast<size_t>(item) * p.most;
    int32_t* to = from + p.most;
    eq = eq0;
    for (int k = w0; k < w1; ++k) {
        const int s = s0 + k * 32 + lane;
        const bool kept = kept_of(s, eq);
        const unsigned is_hole = __ballot_sync(0xffffffffu, s < min(s1, keep) && !kept);
        const unsigned is_mover = __ballot_sync(0xffffffffu, s >= keep && kept);
        const unsigned lower = (1u << lane) - 1;
        if ((is_hole >> lane) & 1u) to[hole + __popc(is_hole & lower)] = s;
        if ((is_mover >> lane) & 1u) from[mover + __popc(is_mover & lower)] = s;
        hole += __popc(is_hole);
        mover += __popc(is_mover);
    }
    if (C > 1) cluster.sync();   // the lists are whole
    else __syncthreads();

    // 3. the moves
    const int row_bytes = p.c.D * (p.c.e4m3 ? 1 : 2);
    const int pieces = row_bytes >> 4;                  // 16-byte pieces of a row: 4, 8 or 16
    const int per_move = 2 * pieces;
    const int lane_of = tid % per_move, slots = C * kThreads / per_move;
    const bool is_v = lane_of >= pieces;
    const int piece = lane_of % pieces;
    uint8_t* pool = is_v ? p.c.v : p.c.k;
    uint8_t* exps = is_v ? p.c.v_exp : p.c.k_exp;
    int bad = 0;
    for (int j = (rank * kThreads + tid) / per_move; j < total; j += slots) {
        const int src = __ldcg(from + j), dst = __ldcg(to + j);
        const int pg_s = page_of(p.c, i, src), pg_d = page_of(p.c, i, dst);
        if (lane_of == 0) {
            mass_out[dst] = __ldcg(mass + src);
            pos_out[dst] = where(src);
        }
        if (pg_s < 0 || pg_d < 0) {
            bad = SDM_DEV_BAD_PAGE;
            continue;
        }
        const size_t head = static_cast<size_t>(g) << p.c.page_shift;
        const size_t rs = pool_row(p.c, pg_s, src) + head, rd = pool_row(p.c, pg_d, dst) + head;
        *reinterpret_cast<uint4*>(pool + rd * row_bytes + piece * 16) =
            *reinterpret_cast<const uint4*>(pool + rs * row_bytes + piece * 16);
        if (p.c.e4m3 && piece == 0) exps[rd] = exps[rs];
    }
    if (bad) set_status(p.dev_status, bad);
    if (C > 1) cluster.sync();   // nobody leaves while its counts are read
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
    while (C < 8 && items * C * 2 <= 2LL * num_sms() && p.stride / (2 * C) >= 2048) C *= 2;
    const long long per = ((p.stride + C - 1) / C + 31) / 32 * 32;
    constexpr int kMost = 48 * 1024;   // keys a CTA can hold
    static const cudaError_t raised =
        cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost * 4);
    if (raised != cudaSuccess) return raised;
    q.room = static_cast<int>(std::min<long long>(per, kMost));
    return launch_cluster(evict_kernel, dim3(static_cast<unsigned>(items * C)), dim3(kThreads), C, q.room * 4, s, q);
}

}  // namespace sdm
