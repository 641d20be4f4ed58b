// attend.cu - attention of packed windows over a paged key/value cache.
//
// One CTA per (request, kv head, 64 rows), a row being one query head of one
// window token (the query heads that share a kv head stand side by side, so
// a tile of keys serves them all).  Tiles of 64 keys pass through shared
// memory as fp32 with the running maximum and sum of the softmax per row:
//     m' = max(m, max_j s_j),  l' = l 2^(m - m') + sum_j 2^(s_j - m'),
//     o' = o 2^(m - m') + sum_j 2^(s_j - m') v_j,   out = o / l.
#include "paged.cuh"

namespace sdm {
namespace {

constexpr int kRows = 64;
constexpr int kKeys = 64;
constexpr int kThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <int D>
struct Smem {
    float q[kRows][D + 4];
    float kv[kKeys][D + 4];
    float p[kRows][kKeys + 4];
    float m[kRows], l[kRows], corr[kRows];
    int page[kKeys];
};

// Whether the row at window position w (position pos) sees token j.
__device__ __forceinline__ bool sees(const AttendParams& p, const Window& w, const uint32_t* bits, int pos, int j) {
    if (p.tree && j >= w.ctx) {
        const int c = j - w.ctx;
        return c < w.n && ((__ldg(bits + (c >> 5)) >> (c & 31)) & 1u);
    }
    return j <= pos && (p.window <= 0 || pos - j < p.window || j < p.sinks);
}

template <int D, bool E4M3>
__device__ __forceinline__ void load_rows(const AttendParams& p, float (*dst)[D + 4], const int* page, bool v, int h,
                                          int j0, int end) {
    for (int t = threadIdx.x; t < kKeys * (D / 8); t += kThreads) {
        const int r = t / (D / 8), c = t % (D / 8);
        float f[8] = {};
        if (j0 + r < end) {
            const size_t row = pool_row(p.c, page[r], j0 + r) + (static_cast<size_t>(h) << p.c.page_shift);
            if constexpr (E4M3) {
                const float s = pow2f(static_cast<int>((v ? p.c.v_exp : p.c.k_exp)[row]) - 127);
                const uint2 x = reinterpret_cast<const uint2*>((v ? p.c.v : p.c.k) + row * D)[c];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 y = f16x2_to_f32x2(
                        e4m3x2_to_f16x2(static_cast<uint16_t>((k < 2 ? x.x : x.y) >> (16 * (k & 1)))));
                    f[2 * k] = y.x * s;
                    f[2 * k + 1] = y.y * s;
                }
            } else {
                const uint4 x = reinterpret_cast<const uint4*>((v ? p.c.v : p.c.k) + row * D * 2)[c];
                const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    f[2 * k] = bf16_bits_to_float(u[k] & 0xffffu);
                    f[2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) dst[r][c * 8 + k] = f[k];
    }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kThreads) attend_kernel(const AttendParams p) {
    extern __shared__ __align__(16) uint8_t raw[];
    Smem<D>& s = *reinterpret_cast<Smem<D>*>(raw);
    pdl_wait();
    pdl_trigger();
    const int i = blockIdx.z, h = blockIdx.y;
    const Window w = window_of(p.cu, p.ctx, i, p.rows, p.max_window, table_tokens(p.c));
    if (w.bad && threadIdx.x == 0) set_status(p.dev_status, w.bad);
    const int M = w.n * p.group, m0 = blockIdx.x * kRows;
    if (m0 >= M) return;
    const int m1 = min(M, m0 + kRows);
    for (int t = threadIdx.x; t < kRows * D; t += kThreads) {
        const int r = t / D, d = t % D, m = m0 + r;
        float x = 0.f;
        if (m < M) {
            const int wp = m / p.group, g = m % p.group;
            x = bf16_bits_to_float(p.q[(w.row0 + wp) * p.q_stride + static_cast<size_t>(h * p.group + g) * D + d]);
        }
        s.q[r][d] = x;
    }
    if (threadIdx.x < kRows) {
        s.m[threadIdx.x] = -INFINITY;
        s.l[threadIdx.x] = 0.f;
    }
    // thread (ty, tx): rows ty * 4 .. + 3; keys tx + 16 c of the scores; dims tx * (D / 16) .. of the output
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float o[4][D / 16] = {};
    const int last = (m1 - 1) / p.group, first = m0 / p.group;
    const int end = p.tree ? w.ctx + w.n : w.ctx + last + 1;
    const int lo = p.window > 0 ? max(0, w.ctx + (p.tree ? 0 : first) - p.window + 1) : 0;
    const float sl = p.scale * kLog2e;
    for (int j0 = 0; j0 < end; j0 += kKeys) {
        if (j0 + kKeys <= lo && j0 >= p.sinks) continue;
        __syncthreads();
        if (threadIdx.x < kKeys) {
            int pg = j0 + threadIdx.x < end ? page_of(p.c, i, j0 + threadIdx.x) : 0;
            if (pg < 0) {
                set_status(p.dev_status, SDM_DEV_BAD_PAGE);
                pg = 0;
            }
            s.page[threadIdx.x] = pg;
        }
        __syncthreads();
        load_rows<D, E4M3>(p, s.kv, s.page, false, h, j0, end);
        __syncthreads();
        float x[4][4] = {};
        for (int d = 0; d < D; ++d) {
            float a[4], b[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) a[r] = s.q[ty * 4 + r][d];
#pragma unroll
            for (int c = 0; c < 4; ++c) b[c] = s.kv[tx + 16 * c][d];
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int c = 0; c < 4; ++c) x[r][c] = fmaf(a[r], b[c], x[r][c]);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int m = m0 + ty * 4 + r;
            const int wp = m / p.group;
            const uint32_t* bits = p.tree ? p.tree + (static_cast<size_t>(i) * p.nodes + min(wp, w.n - 1)) * p.words : nullptr;
            int pos = w.ctx + wp;
            if (p.tree) {
                int n = 0;
                for (int k = 0; k < p.words; ++k) n += __popc(__ldg(bits + k));
                pos = w.ctx + max(0, n - 1);
            }
            float top = -INFINITY;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int j = j0 + tx + 16 * c;
                x[r][c] = (m < M && j < end && sees(p, w, bits, pos, j)) ? x[r][c] * sl : -INFINITY;
                top = fmaxf(top, x[r][c]);
            }
#pragma unroll
            for (int k = 8; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
            const float m_old = s.m[ty * 4 + r];
            const float m_new = fmaxf(m_old, top);
            const float ref = m_new == -INFINITY ? 0.f : m_new;
            float sum = 0.f;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float e = exp2f(x[r][c] - ref);
                s.p[ty * 4 + r][tx + 16 * c] = e;
                sum += e;
            }
#pragma unroll
            for (int k = 8; k > 0; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
            __syncwarp();
            const float corr = exp2f(m_old - ref);
            if (tx == 0) {
                s.m[ty * 4 + r] = m_new;
                s.l[ty * 4 + r] = s.l[ty * 4 + r] * corr + sum;
                s.corr[ty * 4 + r] = corr;
            }
        }
        __syncthreads();
        load_rows<D, E4M3>(p, s.kv, s.page, true, h, j0, end);
        __syncthreads();
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float corr = s.corr[ty * 4 + r];
#pragma unroll
            for (int d = 0; d < D / 16; ++d) o[r][d] *= corr;
        }
        for (int j = 0; j < kKeys; ++j) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float e = s.p[ty * 4 + r][j];
                if (e == 0.f) continue;   // unseen: its value may be anything
#pragma unroll
                for (int d = 0; d < D / 16; ++d) o[r][d] = fmaf(e, s.kv[j][tx + 16 * d], o[r][d]);
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int m = m0 + ty * 4 + r;
        if (m >= M) continue;
        const int wp = m / p.group, g = m % p.group;
        const size_t at = static_cast<size_t>(w.row0 + wp) * p.H + h * p.group + g;
        const float l = s.l[ty * 4 + r];
#pragma unroll
        for (int d = 0; d < D / 16; ++d)
            p.out[at * D + tx + 16 * d] =
                static_cast<uint16_t>(f32x2_to_bf16x2(l == 0.f ? 0.f : o[r][d] / l, 0.f) & 0xffffu);
        if (tx == 0 && p.lse) p.lse[at] = l == 0.f ? -INFINITY : s.m[ty * 4 + r] * kLn2 + logf(l);
    }
}

}  // namespace

size_t attend_workspace(int R, int max_window, int H, int D, int rows, int kv_heads) {
    (void)R;
    (void)max_window;
    (void)H;
    (void)D;
    (void)rows;
    (void)kv_heads;
    return 256;
}

template <int D, bool E4M3>
static cudaError_t launch_one(const AttendParams& p, cudaStream_t s) {
    const int smem = static_cast<int>(sizeof(Smem<D>));
    const cudaError_t e =
        cudaFuncSetAttribute(attend_kernel<D, E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int blocks = static_cast<int>((static_cast<long long>(p.max_window) * p.group + kRows - 1) / kRows);
    return launch_pdl(attend_kernel<D, E4M3>, dim3(blocks, p.c.heads, p.R), dim3(kThreads), smem, s, p);
}

cudaError_t launch_attend(const AttendParams& p, void*, cudaStream_t s) {
    if (p.c.D == 64) return p.c.e4m3 ? launch_one<64, true>(p, s) : launch_one<64, false>(p, s);
    return p.c.e4m3 ? launch_one<128, true>(p, s) : launch_one<128, false>(p, s);
}

}  // namespace sdm
