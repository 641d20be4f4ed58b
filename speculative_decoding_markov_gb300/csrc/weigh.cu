// weigh.cu - the attention weight that every cached token got from a call's
// committed rows, added to what it had.
//
// Mathematics, for token j of a request and kv head g:
//     out_j = (j < ctx ? in_j : 0) + sum over rows p and heads h of g with j
//             visible of exp(scale q_ph . k_j - lse_ph)
// with the log-sum-exp that the attention left.  No maximum is needed: every
// term is a softmax weight, at most 1.
#include <algorithm>

#include "paged.cuh"

namespace sdm {
namespace {

constexpr int kTile = 128;            // keys of a tile, one a thread
constexpr int kRows = 16;             // query rows staged together
constexpr float kLog2e = 1.4426950408889634f;

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

template <int D, bool E4M3>
__global__ void __launch_bounds__(kTile) weigh_kernel(const WeighParams p) {
    __shared__ float q[kRows][D];
    __shared__ float l2[kRows];
    __shared__ int at[kRows];
    pdl_wait();
    pdl_trigger();
    const int i = blockIdx.z, g = blockIdx.y, key0 = blockIdx.x * kTile;
    const Counted w = counted_of(p, i);
    if (w.bad && blockIdx.x == 0 && g == 0 && threadIdx.x == 0) set_status(p.dev_status, w.bad);
    const int n = w.ctx + w.n;
    if (key0 >= n) return;
    const int j = key0 + threadIdx.x;
    float k[D];
    bool held = j < n;
    if (held) {
        int pg = page_of(p.c, i, j);
        if (pg < 0) {
            set_status(p.dev_status, SDM_DEV_BAD_PAGE);
            pg = 0;
        }
        const size_t row = pool_row(p.c, pg, j) + (static_cast<size_t>(g) << p.c.page_shift);
        const float s = E4M3 ? scale_of(__ldg(p.c.k_exp + row)) : 1.f;
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if constexpr (E4M3)
                k[d] = f16x2_to_f32x2(e4m3x2_to_f16x2(p.c.k[row * D + d])).x * s;
            else
                k[d] = bf16_bits_to_float(reinterpret_cast<const uint16_t*>(p.c.k)[row * D + d]);
        }
    }
    float sum = 0.f;
    const int M = w.n * p.group;
    const float c = p.scale * kLog2e;
    for (int m0 = 0; m0 < M; m0 += kRows) {
        __syncthreads();
        for (int t = threadIdx.x; t < kRows * D; t += kTile) {
            const int m = m0 + t / D, wp = m / p.group, h = g * p.group + m % p.group;
            const long long row = m < M ? row_of(p, w, i, wp) : -1;
            q[t / D][t % D] = row >= 0 ? bf16_bits_to_float(p.q[row * p.q_stride + static_cast<size_t>(h) * D + t % D]) : 0.f;
            if (t % D == 0) {
                float z = row >= 0 ? p.lse[row * p.H + h] : -INFINITY;
                at[t / D] = z == -INFINITY ? -1 : w.ctx + wp;      // nothing seen: weighs nothing
                l2[t / D] = z * kLog2e;
                if (m < M && row < 0 && blockIdx.x == 0 && g == 0) set_status(p.dev_status, SDM_DEV_BAD_WINDOW);
            }
        }
        __syncthreads();
        if (!held) continue;
        for (int r = 0; r < min(kRows, M - m0); ++r) {
            const int t = at[r];
            if (j > t || (p.window > 0 && t - j >= p.window && j >= p.sinks)) continue;
            float s = 0.f;
#pragma unroll
            for (int d = 0; d < D; ++d) s = fmaf(q[r][d], k[d], s);
            sum += fast_exp2(fmaf(s, c, -l2[r]));
        }
    }
    if (held) {
        const size_t o = (static_cast<size_t>(i) * p.c.heads + g) * p.stride + j;
        p.mass_out[o] = (j < w.ctx && p.mass ? p.mass[o] : 0.f) + sum;
    }
}

}  // namespace

size_t weigh_workspace(int max_count, int H, int kv_heads) { return 0; }

cudaError_t launch_weigh(const WeighParams& p, void* ws, cudaStream_t s) {
    const long long tokens = std::min<long long>(p.stride, static_cast<long long>(p.c.max_pages) << p.c.page_shift);
    const dim3 grid(static_cast<unsigned>((tokens + kTile - 1) / kTile), p.c.heads, p.R);
    auto k = p.c.D == 128 ? (p.c.e4m3 ? weigh_kernel<128, true> : weigh_kernel<128, false>)
                          : (p.c.e4m3 ? weigh_kernel<64, true> : weigh_kernel<64, false>);
    return launch_pdl(k, grid, dim3(kTile), 0, s, p);
}

}  // namespace sdm
