// cache.cu - the paged key/value cache: writing a window's keys and values
// (quantised to e4m3 as they are written), reading tokens back, and moving a
// tree's accepted path to follow the committed tokens.
//
// All three only move bytes, so each is bounded by HBM at large sizes and by
// one chain of dependent loads (row -> request -> page -> slot) at small ones.
#include <algorithm>

#include "paged.cuh"

namespace sdm {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCommitThreads = 512;     // 32 trees of 65 slots, written and committed: 8.4 us (256: 9.2, 1024: 8.5)

// The windows are looked at apart from the rows, by one block more than the
// rows have (a window that counts as empty need not have a row in use): it
// flags what is wrong with them and returns whether one of them is unsound, in
// which case the rows' own search in cu_seqlens proves nothing and the block
// takes every window's rows itself.  0.4 us of the write and read of 64 windows
// (6.2 us in a graph).
__device__ __forceinline__ bool check_windows(const int32_t* cu, const int32_t* ctx, int R, int rows,
                                              long long tokens, int32_t* dev_status) {
    int bad = 0, unsound = 0;
    for (int i = threadIdx.x; i < R; i += kThreads) {
        const Window w = window_of(cu, ctx, i, rows, 0x7fffffff, tokens);
        bad |= w.bad;
        unsound |= w.n == 0 && (w.bad & SDM_DEV_BAD_WINDOW);
    }
    if (bad) set_status(dev_status, bad);
    return __syncthreads_or(unsound);
}

// One warp per packed row, its loads in flight before the row's slot is
// known.  D / 8 lanes hold one (K or V, head) vector of D elements, 16 bytes
// each, so the maximum of a vector is a shuffle reduction over those lanes.
// e4m3: the smallest scale 2^e with max |x| <= 448 2^e, so that a code's error
// is 2^-4 of its value, or 2^-10 2^e where that is more; scaling is exact.
// 24831 rows of 8 heads x 128 as e4m3: 41 us, 3.7 TB/s, the conversion's 62 %
// of the issue slots beside it; small calls are the chain cu_seqlens -> request
// -> page -> slot (8 us from cold caches for 2080 rows).
template <int D, bool E4M3>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const CacheWriteParams p) {
    constexpr int kLanes = D / 8;           // lanes per vector
    constexpr int kPer = 32 / kLanes;       // vectors per warp pass
    constexpr int kBatch = 4;               // passes whose loads are in flight together
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int sub = lane / kLanes, part = lane % kLanes;
    const int vectors = 2 * p.c.heads;      // K's heads, then V's
    const long long tokens = table_tokens(p.c);
    // row's request: `known`, or (-1) the one that the search gives
    auto write_row = [&](int row, int known) {
        size_t at = 0;
        bool found = false, ok = false;
        for (int v0 = 0; v0 < vectors; v0 += kPer * kBatch) {
            uint4 x[kBatch];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const int vec = v0 + b * kPer + sub;
                const bool is_v = vec >= p.c.heads;
                const uint16_t* src = is_v ? p.v + row * p.v_stride + static_cast<size_t>(vec - p.c.heads) * D
                                           : p.k + row * p.k_stride + static_cast<size_t>(vec) * D;
                x[b] = make_uint4(0, 0, 0, 0);
                if (vec < vectors) x[b] = __ldg(reinterpret_cast<const uint4*>(src) + part);
            }
            if (!found) {
                found = true;
                const int i = known >= 0 ? known : warp_find_request(p.cu, p.R, row);
                const Window w = window_of(p.cu, p.ctx, i, p.rows, 0x7fffffff, tokens);
                if (row >= w.row0 && row < w.row0 + w.n) {
                    const int pos = w.ctx + (row - w.row0);
                    const int pg = page_of(p.c, i, pos);
                    ok = pg >= 0;
                    if (ok) at = pool_row(p.c, pg, pos);
                    else if (lane == 0) set_status(p.dev_status, SDM_DEV_BAD_PAGE);
                }
            }
            if (!ok) break;
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const int vec = v0 + b * kPer + sub;
                const bool is_v = vec >= p.c.heads;
                const int h = is_v ? vec - p.c.heads : vec;
                const size_t r = at + (static_cast<size_t>(h) << p.c.page_shift);
                if constexpr (!E4M3) {
                    if (vec < vectors) reinterpret_cast<uint4*>((is_v ? p.c.v : p.c.k) + r * D * 2)[part] = x[b];
                } else {
                    const uint32_t u[4] = {x[b].x, x[b].y, x[b].z, x[b].w};
                    // the largest finite magnitude, on the bf16 bits
                    uint32_t top = 0;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t lo = u[j] & 0x7fffu, hi = (u[j] >> 16) & 0x7fffu;
                        if (lo < 0x7f80u) top = max(top, lo);
                        if (hi < 0x7f80u) top = max(top, hi);
                    }
#pragma unroll
                    for (int o = kLanes / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                    // max |x| = 1.f 2^(E - 127) <= 448 2^e = 1.75 2^(8 + e)
                    int e = static_cast<int>(top >> 7) - 135 + ((top & 0x7fu) > 0x60u ? 1 : 0);
                    e = min(max(e, kExpLo), kExpHi);
                    const float inv = pow2f(-e);
                    uint32_t code[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float f[4];
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            const float y = bf16_bits_to_float((u[2 * j + (t >> 1)] >> (16 * (t & 1))) & 0xffffu);
                            f[t] = __fmaf_rn(y, inv, y * 0.0f);   // the scaling is exact; an infinity becomes NaN
                        }
                        code[j] = f32x2_to_e4m3x2(f[0], f[1]) |
                                  (static_cast<uint32_t>(f32x2_to_e4m3x2(f[2], f[3])) << 16);
                    }
                    if (vec < vectors) {
                        reinterpret_cast<uint2*>((is_v ? p.c.v : p.c.k) + r * D)[part] = make_uint2(code[0], code[1]);
                        if (part == 0) (is_v ? p.c.v_exp : p.c.k_exp)[r] = static_cast<uint8_t>(e + 127);
                    }
                }
            }
        }
    };
    const int warp = threadIdx.x >> 5, blocks = gridDim.x - 1;
    if (static_cast<int>(blockIdx.x) < blocks) {
        const int n_rows = min(p.rows, __ldg(p.cu + p.R));
        for (int row = blockIdx.x * kWarps + warp; row < n_rows; row += blocks * kWarps) write_row(row, -1);
    } else if (check_windows(p.cu, p.ctx, p.R, p.rows, tokens, p.dev_status)) {
        for (int i = 0; i < p.R; ++i) {
            const Window w = window_of(p.cu, p.ctx, i, p.rows, 0x7fffffff, tokens);
            for (int k = warp; k < w.n; k += kWarps) write_row(w.row0 + k, i);
        }
    }
}

// One warp per output row; D / 8 lanes read 8 elements each of one vector and
// write them as 16 bytes of bf16: code x 2^e is exact in bf16.  46418
// tokens of 8 heads x 128 from e4m3: 50 us, 5.7 TB/s, bound by HBM.
template <int D, bool E4M3>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const CacheReadParams p) {
    constexpr int kLanes = D / 8;
    constexpr int kPer = 32 / kLanes;
    constexpr int kBatch = 4;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int sub = lane / kLanes, part = lane % kLanes;
    const int vectors = 2 * p.c.heads;
    auto read_row = [&](int row, int known) {
        const int i = known >= 0 ? known : warp_find_request(p.cu, p.R, row);
        const Window w = window_of(p.cu, p.first, i, p.rows, 0x7fffffff, 0x7fffffffll);
        if (row < w.row0 || row >= w.row0 + w.n) return;
        const int pos = w.ctx + (row - w.row0);
        const int pg = page_of(p.c, i, pos);
        if (pg < 0 && lane == 0) set_status(p.dev_status, SDM_DEV_BAD_PAGE);
        const size_t at = pg >= 0 ? pool_row(p.c, pg, pos) : 0;
        for (int v0 = 0; v0 < vectors; v0 += kPer * kBatch) {
            uint4 x[kBatch];
            uint2 code[kBatch];
            uint32_t e[kBatch];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const int vec = v0 + b * kPer + sub;
                const bool is_v = vec >= p.c.heads;
                const size_t r = at + (static_cast<size_t>(is_v ? vec - p.c.heads : vec) << p.c.page_shift);
                x[b] = make_uint4(0, 0, 0, 0);
                code[b] = make_uint2(0, 0);
                e[b] = 127;
                if (vec < vectors && pg >= 0) {
                    if constexpr (E4M3) {
                        code[b] = __ldg(reinterpret_cast<const uint2*>((is_v ? p.c.v : p.c.k) + r * D) + part);
                        e[b] = __ldg((is_v ? p.c.v_exp : p.c.k_exp) + r);
                    } else {
                        x[b] = __ldg(reinterpret_cast<const uint4*>((is_v ? p.c.v : p.c.k) + r * D * 2) + part);
                    }
                }
            }
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const int vec = v0 + b * kPer + sub;
                const bool is_v = vec >= p.c.heads;
                const int h = is_v ? vec - p.c.heads : vec;
                if constexpr (E4M3) {
                    const float s = scale_of(e[b]);
                    uint32_t o[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t c2 = (j < 2 ? code[b].x : code[b].y) >> (16 * (j & 1));
                        const float2 f = f16x2_to_f32x2(e4m3x2_to_f16x2(static_cast<uint16_t>(c2)));
                        o[j] = f32x2_to_bf16x2(f.x * s, f.y * s);
                    }
                    x[b] = make_uint4(o[0], o[1], o[2], o[3]);
                }
                if (vec < vectors)
                    reinterpret_cast<uint4*>((is_v ? p.v_out : p.k_out) +
                                             (static_cast<size_t>(row) * p.c.heads + h) * D)[part] = x[b];
            }
        }
    };
    const int warp = threadIdx.x >> 5, blocks = gridDim.x - 1;
    if (static_cast<int>(blockIdx.x) < blocks) {
        const int n_rows = min(p.rows, __ldg(p.cu + p.R));
        for (int row = blockIdx.x * kWarps + warp; row < n_rows; row += blocks * kWarps) read_row(row, -1);
    } else if (check_windows(p.cu, p.first, p.R, p.rows, 0x7fffffffll, p.dev_status)) {
        for (int i = 0; i < p.R; ++i) {
            const Window w = window_of(p.cu, p.first, i, p.rows, 0x7fffffff, 0x7fffffffll);
            for (int k = warp; k < w.n; k += kWarps) read_row(w.row0 + k, i);
        }
    }
}

// One CTA per request: path[0] = the root, path[j + 1] = the child of path[j]
// whose token is out_tok[j]; then row path[j] moves to row j.  The bytes are
// few, so the time is a chain of dependent loads: 8 to 9 us from cold caches for
// 32 trees of 65 slots, 8 heads x 128.  The first warp walks the tree (one ballot per 32
// slots and level), then all threads move the path's rows in order of their
// destination: a batch is loaded whole, then stored.  A source slot path[j]
// is never below its destination j, so a store cannot reach a slot that a
// later batch still reads.
__global__ void __launch_bounds__(kCommitThreads) cache_commit_kernel(const CacheCommitParams p) {
    extern __shared__ int32_t s_tree[];   // parent [N + 1], tok [N + 1], path [B + 1]
    __shared__ int s_len;
    const int S = p.N + 1;
    int32_t* s_parent = s_tree;
    int32_t* s_tok = s_tree + S;
    int32_t* s_path = s_tree + 2 * S;
    const int i = blockIdx.x;
    pdl_wait();
    pdl_trigger();
    for (int c = threadIdx.x; c < S; c += kCommitThreads) {
        s_parent[c] = __ldg(p.parent + static_cast<size_t>(i) * S + c);
        s_tok[c] = __ldg(p.tok + static_cast<size_t>(i) * S + c);
    }
    const int n = min(max(__ldg(p.n_nodes + i), 1), S);
    const int want = min(max(__ldg(p.accept + i), 0), p.B);
    int ctx = __ldg(p.ctx + i);
    int bad = ctx < 0 ? SDM_DEV_BAD_WINDOW : 0;
    ctx = max(ctx, 0);
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int at = 0, len = 0;
        if (lane == 0) s_path[0] = 0;
        while (len < want) {
            const int t = __ldg(p.out_tok + static_cast<size_t>(i) * (p.B + 1) + len);
            int next = -1;
            for (int c0 = at + 1; c0 < n && next < 0; c0 += 32) {
                const int c = c0 + lane;
                const unsigned hit = __ballot_sync(0xffffffffu, c < n && s_parent[c] == at && s_tok[c] == t);
                if (hit) next = c0 + __ffs(hit) - 1;
            }
            if (next < 0) {
                bad |= SDM_DEV_BAD_TOKEN;
                break;
            }
            at = next;
            ++len;
            if (lane == 0) s_path[len] = at;
        }
        for (int j = len + 1 + lane; j <= p.B; j += 32) s_path[j] = -1;
        if (lane == 0) {
            s_len = len;
            if (p.length) p.length[i] = ctx + len + 1;
        }
    }
    __syncthreads();
    const int len = s_len;
    for (int j = threadIdx.x; j <= p.B; j += kCommitThreads) p.path[static_cast<size_t>(i) * (p.B + 1) + j] = s_path[j];
    // 16-byte pieces of a (slot, K or V, head) row, then the scale exponents
    const int row_bytes = p.c.D * (p.c.e4m3 ? 1 : 2);
    const int pieces = row_bytes >> 4;
    const int per_slot = 2 * p.c.heads * (pieces + (p.c.e4m3 ? 1 : 0));
    const long long total = static_cast<long long>(len) * per_slot;   // the root stays where it is
    constexpr int kBatch = 4;
    for (long long t0 = 0; t0 < total; t0 += kCommitThreads * kBatch) {
        uint4 x[kBatch];
        uint8_t* to[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const long long t = t0 + b * kCommitThreads + threadIdx.x;
            to[b] = nullptr;
            if (t >= total) continue;
            const int j = 1 + static_cast<int>(t / per_slot);
            int r = static_cast<int>(t % per_slot);
            const int src = s_path[j];
            if (src == j) continue;
            const bool exps = r >= 2 * p.c.heads * pieces;
            if (exps) r -= 2 * p.c.heads * pieces;
            const int vec = exps ? r : r / pieces;
            const int piece = exps ? 0 : r % pieces;
            const bool is_v = vec >= p.c.heads;
            const int h = is_v ? vec - p.c.heads : vec;
            const long long ps = static_cast<long long>(ctx) + src, pd = static_cast<long long>(ctx) + j;
            const int pg_s = ps <= 0x7fffffffll ? page_of(p.c, i, static_cast<int>(ps)) : -1;
            const int pg_d = pd <= 0x7fffffffll ? page_of(p.c, i, static_cast<int>(pd)) : -1;
            if (pg_s < 0 || pg_d < 0) {
                bad |= SDM_DEV_BAD_PAGE;
                continue;
            }
            const size_t head = static_cast<size_t>(h) << p.c.page_shift;
            const size_t rs = pool_row(p.c, pg_s, static_cast<int>(ps)) + head;
            const size_t rd = pool_row(p.c, pg_d, static_cast<int>(pd)) + head;
            if (exps) {
                uint8_t* base = is_v ? p.c.v_exp : p.c.k_exp;
                x[b].x = base[rs];
                to[b] = base + rd;
            } else {
                uint8_t* base = is_v ? p.c.v : p.c.k;
                x[b] = *reinterpret_cast<const uint4*>(base + rs * row_bytes + piece * 16);
                to[b] = base + rd * row_bytes + piece * 16;
            }
        }
        __syncthreads();
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const long long t = t0 + b * kCommitThreads + threadIdx.x;
            if (!to[b]) continue;
            if (static_cast<int>(t % per_slot) >= 2 * p.c.heads * pieces) *to[b] = static_cast<uint8_t>(x[b].x);
            else *reinterpret_cast<uint4*>(to[b]) = x[b];
        }
        __syncthreads();
    }
    if (bad && (threadIdx.x == 0 || (bad & SDM_DEV_BAD_PAGE))) set_status(p.dev_status, bad);
}

template <typename P>
cudaError_t launch_rows(void (*const (&k)[4])(const P), const P& p, cudaStream_t s) {
    const int blocks = static_cast<int>(std::min<long long>((p.rows + kWarps - 1) / kWarps, 8LL * num_sms()));
    return launch_pdl(k[(p.c.D == 128 ? 2 : 0) + (p.c.e4m3 ? 1 : 0)], dim3(blocks + 1), dim3(kThreads), 0, s, p);
}

}  // namespace

cudaError_t launch_cache_write(const CacheWriteParams& p, cudaStream_t s) {
    static void (*const k[4])(const CacheWriteParams) = {cache_write_kernel<64, false>, cache_write_kernel<64, true>,
                                                         cache_write_kernel<128, false>, cache_write_kernel<128, true>};
    return launch_rows(k, p, s);
}

cudaError_t launch_cache_read(const CacheReadParams& p, cudaStream_t s) {
    static void (*const k[4])(const CacheReadParams) = {cache_read_kernel<64, false>, cache_read_kernel<64, true>,
                                                        cache_read_kernel<128, false>, cache_read_kernel<128, true>};
    return launch_rows(k, p, s);
}

cudaError_t launch_cache_commit(const CacheCommitParams& p, cudaStream_t s) {
    // the limit is the process's, so it is raised once, to what the largest call needs
    constexpr int kMost = (2 * kCommitMost + kCommitMost + 1) * sizeof(int32_t);
    static_assert(kMost <= 224 * 1024, "shared memory");
    static const cudaError_t raised =
        cudaFuncSetAttribute(cache_commit_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    if (raised != cudaSuccess) return raised;
    const size_t smem = (2 * static_cast<size_t>(p.N + 1) + p.B + 1) * sizeof(int32_t);
    return launch_pdl(cache_commit_kernel, dim3(p.R), dim3(kCommitThreads), smem, s, p);
}

}  // namespace sdm
