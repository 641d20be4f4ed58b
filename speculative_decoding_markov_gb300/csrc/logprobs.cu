// logprobs.cu - log probabilities of committed tokens, the distributions'
// entropy, the tokens' ranks and the most probable tokens.
//
// Mathematics, per row z of V logits, c = log2(e) / T and a reference m near
// the row's maximum:  d_v = c z_v - m,  s = sum 2^d,  t = sum d 2^d
//     log p(y) = ln 2 (d_y - log2 s)        H = ln 2 (log2 s - t / s)
// (d <= a few, so H has no cancellation), in one pass over the row, which
// streams through shared memory by bulk copies: every
// thread keeps (m, s, t) of its own elements and moves m only when an element
// exceeds it by more than kLazy.  The listed tokens come from the same pass:
// a thread also keeps its largest element, and the top-th largest of (four a
// warp of) those is a bound that at least `top` elements reach; only the
// threads whose largest reaches it look at their elements again.
//
// What bounds it: 1000 rows of 129280 in fp32 HBM, 5.7 TB/s (90 us); 64 requests
// of 1 to 8 tokens of 151936 in bf16 (290 rows) 29 us, of which the list of 20
// tokens a row is 4 us, the issue of some 9 instructions an element 10 us, and
// the rest the ends of rows that are too few to cover one another; one row 9.6
// us in a graph, a chain of look-ups, sums and the list.
#include <cooperative_groups.h>

#include <algorithm>

#include "device.cuh"
#include "internal.h"

namespace sdm {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTopMost = 32;
constexpr int kStages = 3;             // of the ring that a row streams through
constexpr int kStageBytes = 16384;
constexpr int kCand = 2048;           // listed elements of a CTA
constexpr int kMaxCluster = 8;
constexpr float kLazy = 8.0f;         // in log2 units
constexpr float kLn2 = 0.6931471805599453f;
// A reference's rounding shifts every d of a row alike, by up to 2^-24 of it: no
// matter for d itself, but 2^d has to stay finite.  Rows whose largest c z is
// beyond this are summed with care.
constexpr float kHuge = 1.0e8f;
constexpr float kFar = 1.0e30f;       // a logit beside which log s does not count, and c z may overflow
constexpr float kMaxRef = 3.0e38f;    // references stay finite
constexpr float kLowest = -1.0e30f;   // logits below it have a weight of 0 beside a largest one above -kHuge

struct Part {                          // one CTA's share of a row
    float m, s, t, top;                // reference (scaled), sums, largest logit
    int ahead;                         // elements ahead of the given token
    int n;                             // entries of best
    unsigned long long best[kTopMost];
};

struct Shared {
    float m[kWarps], s[kWarps], t[kWarps], top[kWarps];
    int ahead[kWarps];
    __align__(16) uint32_t maxima[kWarps * 4];
    uint32_t bound;
    int count, ones, wholes, late;
    int one[kThreads], whole[kThreads];
    unsigned long long round[kWarps];
    double sd[kWarps], td[kWarps];
    uint64_t full[kStages], empty[kStages];
    Part part;                         // this CTA's
    Part row;                          // the row's sums
    Part parts[kMaxCluster];           // all CTAs', in the first one
    unsigned long long* cand;          // [kCand], where the ring was
};
static_assert(kCand * 8 <= kStages * kStageBytes && kWarps * 4 >= kTopMost, "lists");

__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y), "f"(z.x), "f"(z.y));
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
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ __nv_bfloat162 pair_of(uint32_t u) { return *reinterpret_cast<__nv_bfloat162*>(&u); }
__device__ __forceinline__ uint32_t bits_of(__nv_bfloat162 x) { return *reinterpret_cast<uint32_t*>(&x); }

// An element's place in the list.  A NaN stands with the elements of -inf,
// whatever its sign and payload: a thread's largest element, which leaves NaN
// out, is then the largest of all of its places, and -inf if it has only NaN.
__device__ __forceinline__ uint32_t place_of(float z) { return ordered_bits(z == z ? z : -INFINITY); }
__device__ __forceinline__ unsigned long long list_key(float z, uint32_t id) {
    return argmax_key(z == z ? z : -INFINITY, id);
}

// Eight logits of a row, from element 8 vec on.
template <bool FP32>
struct Vec {
    uint32_t u[FP32 ? 8 : 4];
    __device__ __forceinline__ void load(const uint8_t* row, int vec) {
        const uint4* src = reinterpret_cast<const uint4*>(row) + (FP32 ? 2 * static_cast<size_t>(vec) : vec);
        set(__ldg(src), FP32 ? __ldg(src + 1) : make_uint4(0, 0, 0, 0));
    }
    __device__ __forceinline__ void load_shared(const uint8_t* stage, int vec) {
        const uint4* src = reinterpret_cast<const uint4*>(stage) + (FP32 ? 2 * vec : vec);
        set(src[0], FP32 ? src[1] : make_uint4(0, 0, 0, 0));
    }
    __device__ __forceinline__ void set(uint4 a, uint4 b) {
        u[0] = a.x, u[1] = a.y, u[2] = a.z, u[3] = a.w;
        if constexpr (FP32) u[4] = b.x, u[5] = b.y, u[6] = b.z, u[7] = b.w;
    }
    __device__ __forceinline__ float at(int j) const {
        if constexpr (FP32) return __uint_as_float(u[j]);
        else return __uint_as_float(j & 1 ? u[j >> 1] & 0xffff0000u : u[j >> 1] << 16);
    }
    __device__ __forceinline__ void set_lowest() {
#pragma unroll
        for (int j = 0; j < (FP32 ? 8 : 4); ++j) u[j] = FP32 ? 0xff800000u : 0xff80ff80u;
    }
    // The largest; a NaN is left out.
    __device__ __forceinline__ float largest() const {
        if constexpr (FP32) {
            float m = at(0);
#pragma unroll
            for (int j = 1; j < 8; ++j) m = fmaxf(m, at(j));
            return m;
        } else {
            const uint32_t m = bits_of(__hmax2(__hmax2(pair_of(u[0]), pair_of(u[1])), __hmax2(pair_of(u[2]), pair_of(u[3]))));
            return fmaxf(bf16_bits_to_float(m & 0xffffu), bf16_bits_to_float(m >> 16));
        }
    }
    // Elements below kLowest, which weigh nothing, as that (finite: 0 d = 0); a NaN stays.
    __device__ __forceinline__ void raise() {
        if constexpr (FP32) {
#pragma unroll
            for (int j = 0; j < 8; ++j) u[j] = __float_as_uint(max_nan(at(j), kLowest));
        } else {
            const __nv_bfloat162 low = __float2bfloat162_rn(kLowest);
#pragma unroll
            for (int j = 0; j < 4; ++j) u[j] = bits_of(__hmax2_nan(pair_of(u[j]), low));
        }
    }
    // Adds how many exceed x, or (EQUAL) reach it: bf16 counts in both halves of
    // a register, exact to 256.
    template <bool EQUAL>
    __device__ __forceinline__ void above(float x, int& n, __nv_bfloat162& halves) const {
        if constexpr (FP32) {
#pragma unroll
            for (int j = 0; j < 8; ++j) n += EQUAL ? at(j) >= x : at(j) > x;
        } else {
            const __nv_bfloat162 y = __float2bfloat162_rn(x);   // x is one of the row's: exact
#pragma unroll
            for (int j = 0; j < 4; ++j)
                halves = __hadd2(halves, EQUAL ? __hge2(pair_of(u[j]), y) : __hgt2(pair_of(u[j]), y));
        }
    }
};

template <int N>
__device__ __forceinline__ float largest_of(const Vec<true> (&x)[N]) {
    float m = x[0].largest();
#pragma unroll
    for (int k = 1; k < N; ++k) m = fmaxf(m, x[k].largest());
    return m;
}
template <int N>
__device__ __forceinline__ float largest_of(const Vec<false> (&x)[N]) {
    __nv_bfloat162 m = pair_of(x[0].u[0]);
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) m = __hmax2(m, pair_of(x[k].u[j]));
    return fmaxf(__uint_as_float(bits_of(m) << 16), __uint_as_float(bits_of(m) & 0xffff0000u));
}

// (s, t) of a reference m, for the reference `to` >= m.  A factor of zero ends
// what may be infinite beside it.
__device__ __forceinline__ void move_to(float& m, float& s, float& t, float to) {
    const float k = m - to, a = fast_exp2(k);
    t = a == 0.f ? 0.f : a * (t + k * s);
    s = a != 0.f ? s * a : s != s ? s : 0.f;
    m = to;
}

// The sums of a warp's lanes (or of every 2^n neighbours, n steps), in a fixed order.
template <int LANES>
__device__ __forceinline__ void join_lanes(float& m, float& s, float& t, float& top, int& ahead) {
    float to = m;
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, o));
    move_to(m, s, t, to);
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, o);
        t += __shfl_xor_sync(0xffffffffu, t, o);
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        ahead += __shfl_xor_sync(0xffffffffu, ahead, o);
    }
}

// The largest key below `below` of elements [v0, v1) (in vectors), by the whole CTA.
template <bool FP32>
__device__ unsigned long long next_key(const uint8_t* row, int v0, int v1, unsigned long long below, Shared& sh) {
    unsigned long long best = 0;
    for (int v = v0 + threadIdx.x; v < v1; v += kThreads) {
        Vec<FP32> x;
        x.load(row, v);
        for (int j = 0; j < 8; ++j) {
            const unsigned long long k = list_key(x.at(j), 8 * v + j);
            if (k < below) best = umax64(best, k);
        }
    }
    best = warp_max_u64(best);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh.round[threadIdx.x >> 5] = best;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) best = umax64(best, sh.round[w]);
    return best;
}

// A thread's largest element, the stage it is in, and the largest of its other
// stages; without elements all are 0, below any key.
struct Largest {
    uint32_t key, next;
    int stage;
};

// Lists the elements that reach `bound` (`strict`: exceed it), which are among
// those of the threads whose largest one does, mostly in one stage of theirs:
// these stages' vectors, or all of such a thread's, are looked at by all.
template <bool FP32>
__device__ __forceinline__ void list_candidates(const uint8_t* row, int v0, int v1, const Largest& mine, uint32_t bound,
                                                bool strict, Shared& sh) {
    constexpr int kOwn = kStageBytes / (FP32 ? 32 : 16) / kThreads;   // a thread's vectors of a stage
    const uint32_t from = strict ? bound + 1 : bound;
    if (threadIdx.x == 0) sh.count = sh.ones = sh.wholes = 0;
    __syncthreads();
    if (mine.key >= from) {
        if (mine.next >= from) sh.whole[atomicAdd(&sh.wholes, 1)] = static_cast<int>(threadIdx.x);
        else sh.one[atomicAdd(&sh.ones, 1)] = mine.stage * kThreads * kOwn + static_cast<int>(threadIdx.x);
    }
    __syncthreads();
    const int per = (v1 - v0 + kThreads - 1) / kThreads, ones = sh.ones * kOwn, all = ones + sh.wholes * per;
    for (int k = threadIdx.x; k < all; k += kThreads) {
        int v;
        if (k < ones) {
            v = v0 + sh.one[k / kOwn] + (k % kOwn) * kThreads;
        } else {
            const int f = (k - ones) / per;
            v = v0 + sh.whole[f] + (k - ones - f * per) * kThreads;
        }
        if (v >= v1) continue;
        Vec<FP32> x;
        x.load(row, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float z = x.at(j);
            if (place_of(z) >= from) {
                const int at = atomicAdd(&sh.count, 1);
                if (at < kCand) sh.cand[at] = list_key(z, 8 * v + j);
            }
        }
    }
    __syncthreads();
}

// The `top` largest keys of the CTA's elements, in order, into sh.part.best.
template <bool FP32>
__device__ void pick_top(const uint8_t* row, int v0, int v1, const Largest& mine, int top, Shared& sh) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n_out = min(top, 8 * (v1 - v0));
    // four largest of the warp's maxima
    uint32_t left = mine.key;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const uint32_t w = __reduce_max_sync(0xffffffffu, left);
        const unsigned who = __ballot_sync(0xffffffffu, left == w);
        if (lane == __ffs(who) - 1) left = 0;
        if (lane == 0) sh.maxima[warp * 4 + r] = w;
    }
    if (threadIdx.x == 0) sh.bound = 0;
    __syncthreads();
    if (threadIdx.x < kWarps * 4) {
        const uint32_t x = sh.maxima[threadIdx.x];
        const uint4* all = reinterpret_cast<const uint4*>(sh.maxima);
        int before = 0;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            const uint4 y = all[k];
            const int at = threadIdx.x - 4 * k;   // an equal one before it counts
            before += (y.x > x || (y.x == x && at > 0)) + (y.y > x || (y.y == x && at > 1)) +
                      (y.z > x || (y.z == x && at > 2)) + (y.w > x || (y.w == x && at > 3));
        }
        if (before == top - 1) sh.bound = x;
    }
    const int whole = (v1 - v0) / 32;   // warps whose threads all have elements, up to kWarps; then some of the next
    if (whole < kWarps && 4 * whole + min(4, v1 - v0 - 32 * whole) < top) {
        // a short row, whose warps have fewer than `top` such maxima: the top-th
        // largest of all threads' (7729 rows of 1200, 32 listed: 169 us; 2293 with
        // all elements listed and ranked)
        uint32_t* all = reinterpret_cast<uint32_t*>(sh.one);
        all[threadIdx.x] = mine.key;
        __syncthreads();
        int before = 0;
#pragma unroll 8
        for (int k = 0; k < kThreads; ++k) before += all[k] > mine.key || (all[k] == mine.key && k < static_cast<int>(threadIdx.x));
        if (before == top - 1) sh.bound = mine.key;
    }
    __syncthreads();
    const uint32_t bound = sh.bound;
    list_candidates<FP32>(row, v0, v1, mine, bound, false, sh);
    int n = sh.count;
    if (n > kCand) {
        // more reach the bound than fit: those that exceed it, then its lowest ids
        __syncthreads();
        list_candidates<FP32>(row, v0, v1, mine, bound, true, sh);
        n = sh.count;
        if (n <= kCand - kThreads) {
            for (int base = v0; base < v1 && n < n_out; base += kThreads) {
                const int v = base + threadIdx.x;
                Vec<FP32> x;
                uint32_t hit = 0;
                if (v < v1) {
                    x.load(row, v);
#pragma unroll
                    for (int j = 0; j < 8; ++j) hit |= static_cast<uint32_t>(place_of(x.at(j)) == bound) << j;
                }
                // their places, in the order of the ids
                int incl = __popc(hit);
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += y;
                }
                __syncthreads();
                if (lane == 31) sh.ahead[warp] = incl;
                __syncthreads();
                int at = n + incl - __popc(hit), all = 0;
                for (int w = 0; w < kWarps; ++w) {
                    if (w < warp) at += sh.ahead[w];
                    all += sh.ahead[w];
                }
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if ((hit >> j) & 1u) {
                        if (at < n_out) sh.cand[at] = list_key(x.at(j), 8 * v + j);
                        ++at;
                    }
                n = min(n + all, n_out);
            }
            __syncthreads();
        } else {   // one pass a rank
            unsigned long long below = ~0ull;
            for (int r = 0; r < n_out; ++r) {
                below = next_key<FP32>(row, v0, v1, below, sh);
                if (threadIdx.x == 0) sh.part.best[r] = below;
            }
            if (threadIdx.x == 0) sh.part.n = n_out;
            __syncthreads();
            return;
        }
    }
    for (int a = threadIdx.x; a < n; a += kThreads) {
        const unsigned long long k = sh.cand[a];
        int before = 0;
        for (int b = 0; b < n; ++b) before += sh.cand[b] > k;
        if (before < n_out) sh.part.best[before] = k;
    }
    if (threadIdx.x == 0) sh.part.n = n_out;
    __syncthreads();
}

// A cluster of CTAs per row; each takes an equal share of it.
template <bool FP32>
__global__ void __launch_bounds__(kThreads, 4) logprobs_kernel(const LogprobParams p) {
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ Shared sh;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x < kStages) {
        mbar_init(&sh.full[threadIdx.x], 1);
        mbar_init(&sh.empty[threadIdx.x], kWarps);
    }
    if (threadIdx.x == 0) {
        sh.late = 0;
        sh.cand = reinterpret_cast<unsigned long long*>(ring);
    }
    fence_mbar_init();
    pdl_wait();
    pdl_trigger();
    cg::cluster_group cluster = cg::this_cluster();
    const int C = cluster.num_blocks(), rank = cluster.block_rank();
    const int item = blockIdx.x / C, i = item / p.W, pos = item - i * p.W;

    // the row, or nothing (its look-ups are independent loads)
    int n = p.n ? __ldg(p.n + i) : p.W;
    const long long first = __ldg(p.cu + i), end = __ldg(p.cu + i + 1);
    const int off = p.path ? __ldg(p.path + item) : pos;
    int tok = __ldg(p.tok + item);
    int bad = 0;
    if (n < 0 || n > p.W) {
        n = min(max(n, 0), p.W);
        bad = SDM_DEV_BAD_WINDOW;
    }
    if (!p.n) n = static_cast<int>(min(static_cast<long long>(n), max(end - first, 0ll)));
    bool live = pos < n;
    const long long r = first + off;
    if (live) {
        if (first < 0 || off < 0 || r >= end) bad |= SDM_DEV_BAD_WINDOW, live = false;
        else if (r >= p.rows) bad |= SDM_DEV_CAPACITY, live = false;
    }
    const bool known = static_cast<unsigned>(tok) < static_cast<unsigned>(p.V);
    if (live && !known) bad |= SDM_DEV_BAD_TOKEN;
    if (bad && rank == 0 && threadIdx.x == 0) set_status(p.dev_status, bad);
    if (!live) return;   // the whole cluster
    if (!known) tok = 0;

    const uint8_t* row = static_cast<const uint8_t*>(p.target) + static_cast<size_t>(r) * p.V * (FP32 ? 4 : 2);
    const int vecs = p.V / 8;
    const int v0 = static_cast<int>(static_cast<long long>(vecs) * rank / C);
    const int v1 = static_cast<int>(static_cast<long long>(vecs) * (rank + 1) / C);
    const float c = p.scale;
    // The row's share streams through a ring of stages, copied by one thread.
    constexpr int kVecBytes = FP32 ? 32 : 16, kVecs = kStageBytes / kVecBytes;
    const uint8_t* share = row + static_cast<size_t>(v0) * kVecBytes;
    const int vectors = v1 - v0, stages = (vectors + kVecs - 1) / kVecs;
    auto copy = [&](int st) {   // by thread 0
        const int bytes = min(kVecs, vectors - st * kVecs) * kVecBytes;
        mbar_arrive_expect_tx(&sh.full[st % kStages], bytes);
        bulk_load(ring + (st % kStages) * kStageBytes, share + static_cast<size_t>(st) * kStageBytes, bytes,
                  &sh.full[st % kStages]);
    };
    __syncthreads();   // the barriers are set up
    int sent = min(stages, kStages);   // stages copied (thread 0)
    if (threadIdx.x == 0)
        for (int st = 0; st < sent; ++st) copy(st);

    float said = 0.f;
    if (known)
        said = FP32 ? __ldg(reinterpret_cast<const float*>(row) + tok)
                    : bf16_bits_to_float(__ldg(reinterpret_cast<const uint16_t*>(row) + tok));

    float m = -kMaxRef, top = -INFINITY, next = -INFINITY;   // the largest element; of the other stages than top_in
    int top_in = 0;
    float2 s2 = make_float2(0.f, 0.f), t2 = make_float2(0.f, 0.f);
    int ahead = 0;
    __nv_bfloat162 halves = __float2bfloat162_rn(0.f);
    auto flush = [&]() {
        ahead += static_cast<int>(__low2float(halves) + __high2float(halves));
        halves = __float2bfloat162_rn(0.f);
    };
    const int said_in = tok >> 3;        // the vector that holds the token
    for (int st = 0; st < stages; ++st) {
        // one answer a warp: a lane that gave up by itself would leave the loop, and the others
        // would wait for it
        if (!__all_sync(0xffffffffu, mbar_wait(&sh.full[st % kStages], (st / kStages) & 1))) {
            sh.late = 1;
            break;
        }
        const uint8_t* stage = ring + (st % kStages) * kStageBytes;
        // The thread's vectors of the stage together: one look at their largest
        // element decides on the reference and on the comparisons with the
        // given token (most stages have none that reaches it).
        constexpr int kOwn = kVecs / kThreads;
        const int at = v0 + st * kVecs + threadIdx.x;
        Vec<FP32> x[kOwn];
#pragma unroll
        for (int k = 0; k < kOwn; ++k) {
            x[k].set_lowest();
            if (at + k * kThreads < v1) x[k].load_shared(stage, k * kThreads + threadIdx.x);
        }
        const float sm = largest_of(x);
        next = fmaxf(next, fminf(sm, top));
        if (sm > top) {
            top = sm;
            top_in = st;
        }
        if (sm >= said) {
#pragma unroll
            for (int k = 0; k < kOwn; ++k) {
                const int v = at + k * kThreads;
                if (v >= v1) continue;   // filled up with -inf, which a masked token's logit equals
                if (v < said_in) x[k].template above<true>(said, ahead, halves);
                else x[k].template above<false>(said, ahead, halves);
                if (v == said_in)
                    for (int j = 0; j < (tok & 7); ++j) ahead += x[k].at(j) == said;
            }
        }
        if (sm * c > m + kLazy) {
            float s = s2.x + s2.y, t = t2.x + t2.y;
            move_to(m, s, t, fminf(sm * c, kMaxRef));
            s2 = make_float2(s, 0.f);
            t2 = make_float2(t, 0.f);
        }
#pragma unroll
        for (int k = 0; k < kOwn; ++k) {
            x[k].raise();
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const float2 d = fma2(make_float2(x[k].at(j), x[k].at(j + 1)), make_float2(c, c), make_float2(-m, -m));
                const float2 e = make_float2(fast_exp2(d.x), fast_exp2(d.y));
                s2 = add2(s2, e);
                t2 = fma2(e, d, t2);
            }
        }
        if (!FP32 && st % 8 == 7) flush();   // a stage adds at most 16 to a half
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.empty[st % kStages]);
        // the stage before this one is free, or about to be
        if (threadIdx.x == 0 && st > 0 && st - 1 + kStages < stages) {
            if (mbar_wait(&sh.empty[(st - 1) % kStages], ((st - 1) / kStages) & 1)) {
                copy(st - 1 + kStages);
                sent = st + kStages;
            } else {
                sh.late = 1;
            }
        }
        __syncwarp();
    }
    flush();
    Largest mine = {0, 0, top_in};
    if (static_cast<int>(threadIdx.x) < vectors) mine.key = max(ordered_bits(top), 1u), mine.next = ordered_bits(next);

    // the CTA's sums, in the order of lanes and warps
    float s = s2.x + s2.y, t = t2.x + t2.y;
    join_lanes<32>(m, s, t, top, ahead);
    if (lane == 0) {
        sh.m[warp] = m;
        sh.s[warp] = s;
        sh.t[warp] = t;
        sh.top[warp] = top;
        sh.ahead[warp] = ahead;
    }
    __syncthreads();
    if (sh.late && threadIdx.x == 0) {   // a wait's limit: what follows is not to be trusted, and ends
        set_status(p.dev_status, SDM_DEV_TIMEOUT);
        for (int st = max(0, sent - kStages); st < sent; ++st) mbar_wait(&sh.full[st % kStages], (st / kStages) & 1);
    }
    if (warp == 0) {
        const int w = lane & (kWarps - 1);
        m = sh.m[w], s = sh.s[w], t = sh.t[w], top = sh.top[w], ahead = sh.ahead[w];
        join_lanes<kWarps>(m, s, t, top, ahead);
        if (lane == 0) {
            Part& q = sh.part;
            q.m = m, q.s = s, q.t = t, q.top = top, q.ahead = ahead, q.n = 0;
        }
    }
    __syncthreads();
    if (p.top > 0 && v1 > v0) pick_top<FP32>(row, v0, v1, mine, p.top, sh);
    // the shares of a row in every CTA of its cluster, joined by all alike
    if (C > 1) {
        cluster.sync();
        constexpr int kWords = sizeof(Part) / 4;
        for (int k = threadIdx.x; k < C * kWords; k += kThreads)
            reinterpret_cast<uint32_t*>(sh.parts)[k] =
                reinterpret_cast<const uint32_t*>(cluster.map_shared_rank(&sh.part, k / kWords))[k % kWords];
        __syncthreads();
    }
    if (warp == 0) {
        // lanes past the cluster's CTAs add nothing
        const Part& q = C > 1 ? sh.parts[lane & (C - 1)] : sh.part;
        const bool mine = lane < C;
        m = q.m, s = mine ? q.s : 0.f, t = mine ? q.t : 0.f, top = q.top, ahead = mine ? q.ahead : 0;
        if (C > 1) join_lanes<kMaxCluster>(m, s, t, top, ahead);
        if (lane == 0) sh.row.m = m, sh.row.s = s, sh.row.t = t, sh.row.top = top, sh.row.ahead = ahead;
    }
    __syncthreads();
    const Part& row_part = sh.row;
    const float M = row_part.top;
    float S = row_part.s, T = row_part.t;
    const float ref = row_part.m;
    // a row of logits whose products with c leave fp32: summed again in fp64,
    // relative to its largest (the type's lowest value in every place is one)
    const bool careful = fabsf(M) * c >= kHuge && fabsf(M) < INFINITY && S == S;
    const double cd = static_cast<double>(p.inv_t);
    if (careful) {
        double sd = 0, td = 0;
        for (int v = v0 + threadIdx.x; v < v1; v += kThreads) {
            Vec<FP32> x;
            x.load(row, v);
            for (int j = 0; j < 8; ++j) {
                const double d = (static_cast<double>(x.at(j)) - M) * cd;
                const double e = exp(d);
                sd += e;
                if (e > 0) td += e * d;
            }
        }
        for (int o = 16; o > 0; o >>= 1) {
            sd += __shfl_xor_sync(0xffffffffu, sd, o);
            td += __shfl_xor_sync(0xffffffffu, td, o);
        }
        if (lane == 0) sh.sd[warp] = sd, sh.td[warp] = td;
        __syncthreads();
        if (threadIdx.x == 0)
            for (int w = 1; w < kWarps; ++w) sh.sd[0] += sh.sd[w], sh.td[0] += sh.td[w];
        if (C > 1) cluster.sync();
        else __syncthreads();
        sd = td = 0;
        for (int k = 0; k < C; ++k) {
            sd += C > 1 ? *cluster.map_shared_rank(&sh.sd[0], k) : sh.sd[0];
            td += C > 1 ? *cluster.map_shared_rank(&sh.td[0], k) : sh.td[0];
        }
        S = static_cast<float>(sd);
        T = static_cast<float>(td);
    }
    // log p of a logit of the row
    auto logp = [&](float z) {
        if (careful) return static_cast<float>((static_cast<double>(z) - M) * cd - log(static_cast<double>(S)));
        if (fabsf(M) == INFINITY && S == S) return z - M;   // -inf beside +inf, else NaN
        if (fabsf(z) * c >= kFar && S == S) return static_cast<float>((static_cast<double>(z) - M) * cd);
        return kLn2 * (fmaf(z, c, -ref) - log2f(S));
    };
    if (rank == 0 && threadIdx.x == 0) {
        p.logp[item] = known ? logp(said) : -INFINITY;
        if (p.entropy) {
            float h = careful ? logf(S) - T / S : kLn2 * (log2f(S) - T / S);
            if (fabsf(M) == INFINITY) h = __int_as_float(0x7fffffff);
            p.entropy[item] = h;
        }
        if (p.rank) p.rank[item] = known ? row_part.ahead : p.V;
    }
    if (p.top > 0) {
        // a listed token's place: how many of all CTAs' come before it.  The
        // CTAs take turns by their entries.
        for (int a = rank * kThreads + threadIdx.x; a < C * kTopMost; a += C * kThreads) {
            const Part& own = C > 1 ? sh.parts[a / kTopMost] : sh.part;
            if (a % kTopMost >= own.n) continue;
            const unsigned long long k = own.best[a % kTopMost];
            int before = 0;
            for (int b = 0; b < C; ++b) {
                const Part& o = C > 1 ? sh.parts[b] : sh.part;
                for (int e = 0; e < o.n; ++e) before += o.best[e] > k;
            }
            if (before < p.top) {
                const size_t at = static_cast<size_t>(item) * p.top + before;
                const int id = static_cast<int>(key_token(k));
                p.top_tok[at] = id;
                p.top_logp[at] = logp(key_value(k));
            }
        }
    }
    if (C > 1) cluster.sync();   // nobody leaves while its share is read
}

}  // namespace

cudaError_t launch_logprobs(const LogprobParams& p, cudaStream_t s) {
    const long long items = static_cast<long long>(p.R) * p.W;
    // few rows: several SMs a row, as long as each has some thousand elements
    // and the grid stays within two rounds of four blocks an SM (64 requests of
    // 1 to 8 in 512 places: 28.5 us with two blocks a row, 39.6 with one; up
    // to 16 rounds 50)
    int C = 1;
    while (C < kMaxCluster && items * C * 2 <= 8LL * num_sms() && p.V / (2 * C) >= 4096) C *= 2;
    constexpr int kRing = kStages * kStageBytes;
    static SmemLimit limits[2];
    const auto kernel = p.fp32 ? logprobs_kernel<true> : logprobs_kernel<false>;
    const cudaError_t raised = limits[p.fp32 ? 1 : 0].raise(kernel, kRing);
    if (raised != cudaSuccess) return raised;
    return launch_cluster(kernel, dim3(static_cast<unsigned>(items * C)), dim3(kThreads), C, kRing, s, p);
}

}  // namespace sdm
