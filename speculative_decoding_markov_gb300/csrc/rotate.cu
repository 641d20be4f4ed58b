// rotate.cu - queries and keys normalised per head and rotated by their
// positions, the keys and values written into the paged cache on the way.
//
// Mathematics, per head vector x of D elements:
//     y = x rsqrt(mean(x^2) + eps) weight          (no weight: y = x)
//     (a, b) -> (a cos t - b sin t, b cos t + a sin t),  t = position freq_j
// for the pairs j < rot / 2: elements (j, j + rot / 2), or (2 j, 2 j + 1) if
// interleaved; elements from rot on pass.  Everything is fp32 and rounded to
// bf16 once, but the angle: at positions of 10^5 a fp32 product is off by
// 0.01 rad, so the turns position freq / 2 pi are reduced in fp64.
#include <algorithm>

#include "paged.cuh"

namespace sdm {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// What becomes of a section's vectors.
enum { TO_ROWS = 0, TO_CACHE = 1, TO_CACHE_E4M3 = 2 };

// The lane's two pieces of 4 elements of every vector: a pair's two elements
// are one lane's, so the same 4 angles serve every vector, and nothing but the
// sum of squares crosses lanes.
struct Lane {
    int sub, l;            // vector of a pass, lane of the vector
    int r0, r1;            // pieces of a rotated vector
    bool turns;
};

// One row's vectors first .. last - 1 of queries, keys or values (PLAIN): D / 8
// lanes a vector, kBatch passes of the warp loaded while the kBatch before them
// are worked on.
template <int D, bool INTER, bool PLAIN, int TO, int kBatch>
__device__ __forceinline__ void section(const Lane& n, const uint16_t* src, int first, int last, const float* weight,
                                        float eps, const float (&cs)[4], const float (&sn)[4], uint8_t* dst,
                                        size_t head_bytes, uint8_t* exps, size_t head_rows, bool put) {
    constexpr int kLanes = D / 8, kPer = 32 / kLanes;
    const int p0 = PLAIN ? 2 * n.l : n.r0, p1 = PLAIN ? 2 * n.l + 1 : n.r1;
    float w[8];
    if (!PLAIN && weight) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(weight) + p0);
        const float4 b = __ldg(reinterpret_cast<const float4*>(weight) + p1);
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    }
    uint2 x[2][kBatch][2];
    const uint2* s2 = reinterpret_cast<const uint2*>(src);   // not by the read-only path: the outputs may be the inputs
    auto load = [&](int v0, uint2 (&to)[kBatch][2]) {
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int vec = v0 + b * kPer + n.sub;
            to[b][0] = to[b][1] = make_uint2(0, 0);
            if (vec < last) {
                to[b][0] = s2[vec * (D / 4) + p0];
                to[b][1] = s2[vec * (D / 4) + p1];
            }
        }
    };
    auto work = [&](int v0, const uint2 (&from)[kBatch][2]) {
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int vec = v0 + b * kPer + n.sub;
            uint32_t u[4] = {from[b][0].x, from[b][0].y, from[b][1].x, from[b][1].y};
            if constexpr (!PLAIN) {
                float f[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = bf16_bits_to_float((u[j >> 1] >> (16 * (j & 1))) & 0xffffu);
                if (weight) {
                    float sum = 0.f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum = fmaf(f[j], f[j], sum);
#pragma unroll
                    for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    const float inv = rsqrtf(fmaf(sum, 1.0f / D, eps));
#pragma unroll
                    for (int j = 0; j < 8; ++j) f[j] *= inv * w[j];
                }
                if (n.turns) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float& a = f[INTER ? 2 * j : j];
                        float& c = f[INTER ? 2 * j + 1 : j + 4];
                        const float a0 = a, c0 = c;
                        a = a0 * cs[j] - c0 * sn[j];
                        c = c0 * cs[j] + a0 * sn[j];
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) u[j] = f32x2_to_bf16x2(f[2 * j], f[2 * j + 1]);
            }
            if constexpr (TO == TO_CACHE_E4M3) {
                const int e = e4m3_exponent<kLanes>(u);
                const uint2 code = e4m3_codes(u, e);
                if (put && vec < last) {
                    uint32_t* to = reinterpret_cast<uint32_t*>(dst + vec * head_bytes);
                    to[p0] = code.x;
                    to[p1] = code.y;
                    if (n.l == 0) exps[vec * head_rows] = static_cast<uint8_t>(e + 127);
                }
            } else if (put && vec < last) {
                uint2* to = reinterpret_cast<uint2*>(dst + vec * head_bytes);
                to[p0] = make_uint2(u[0], u[1]);
                to[p1] = make_uint2(u[2], u[3]);
            }
        }
    };
    constexpr int kStep = kPer * kBatch;
    load(first, x[0]);
    for (int v0 = first; v0 < last; v0 += 2 * kStep) {
        if (v0 + kStep < last) load(v0 + kStep, x[1]);
        work(v0, x[0]);
        if (v0 + kStep >= last) break;
        if (v0 + 2 * kStep < last) load(v0 + 2 * kStep, x[0]);
        work(v0 + kStep, x[1]);
    }
}

// A warp takes a row, or one of `parts` equal shares of its vectors (query
// heads, key heads and, with a cache, value heads).
template <int D, bool INTER, int TO>
__global__ void __launch_bounds__(kThreads) rotate_kernel(const RotateParams p) {
    constexpr int kLanes = D / 8, kBatch = 2;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int heads = p.H + p.G, vectors = heads + (TO == TO_ROWS ? 0 : p.G);
    const long long tokens = TO == TO_ROWS ? static_cast<long long>(kMaxTokens) : table_tokens(p.c);
    Lane n;
    n.sub = lane / kLanes;
    n.l = lane % kLanes;
    const int half = p.rot / 8;             // pieces of a half; lanes that rotate
    n.turns = n.l < half;
    n.r0 = INTER ? 2 * n.l : n.turns ? n.l : 2 * half + 2 * (n.l - half);
    n.r1 = INTER ? 2 * n.l + 1 : n.turns ? n.l + half : n.r0 + 1;

    auto do_row = [&](int row, int part, int known) {
        const int v_from = static_cast<int>(static_cast<long long>(vectors) * part / p.parts);
        const int v_to = static_cast<int>(static_cast<long long>(vectors) * (part + 1) / p.parts);
        const int i = known >= 0 ? known : warp_find_request(p.cu, p.R, row);
        const Window w = window_of(p.cu, p.ctx, i, p.rows, 0x7fffffff, tokens);
        if (row < w.row0 || row >= w.row0 + w.n) return;
        const int off = row - w.row0;
        const long long first = p.start ? __ldg(p.start + i) : w.ctx;
        const double pos = static_cast<double>(first + (p.row_pos ? __ldg(p.row_pos + row) : off));
        size_t at = 0;
        bool held = false;
        if constexpr (TO != TO_ROWS) {
            const int pg = page_of(p.c, i, w.ctx + off);
            held = pg >= 0;
            if (held) at = pool_row(p.c, pg, w.ctx + off);
            else if (lane == 0) set_status(p.dev_status, SDM_DEV_BAD_PAGE);
        }
        float cs[4], sn[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            cs[j] = 1.f;
            sn[j] = 0.f;
            if (n.turns) {
                constexpr double kInv2Pi = 0.15915494309189533577;
                const double t = pos * __ldg(p.freq + 4 * n.l + j) * kInv2Pi;
                sincospif(2.0f * static_cast<float>(t - rint(t)), &sn[j], &cs[j]);
            }
        }
        if (v_from < p.H)
            section<D, INTER, false, TO_ROWS, kBatch>(n, p.q + row * p.q_stride, v_from, min(v_to, p.H), p.q_weight, p.eps,
                                                      cs, sn, reinterpret_cast<uint8_t*>(p.q_out + row * p.q_out_stride),
                                                      2 * D, nullptr, 0, true);
        const int k_from = max(v_from - p.H, 0), k_to = min(v_to - p.H, p.G);
        const size_t slots = static_cast<size_t>(1) << p.c.page_shift;   // pool rows from head to head
        constexpr int kRow = TO == TO_CACHE_E4M3 ? D : 2 * D;
        if (k_from < k_to) {
            if constexpr (TO == TO_ROWS)
                section<D, INTER, false, TO, kBatch>(n, p.k + row * p.k_stride, k_from, k_to, p.k_weight, p.eps, cs, sn,
                                                     reinterpret_cast<uint8_t*>(p.k_out + row * p.k_out_stride), 2 * D,
                                                     nullptr, 0, true);
            else
                section<D, INTER, false, TO, kBatch>(n, p.k + row * p.k_stride, k_from, k_to, p.k_weight, p.eps, cs, sn,
                                                     p.c.k + at * kRow, slots * kRow, p.c.k_exp + at, slots, held);
        }
        if constexpr (TO != TO_ROWS) {
            const int x_from = max(v_from - heads, 0), x_to = v_to - heads;
            if (x_from < x_to)
                section<D, INTER, true, TO, kBatch>(n, p.v + row * p.v_stride, x_from, x_to, nullptr, 0.f, cs, sn,
                                                    p.c.v + at * kRow, slots * kRow, p.c.v_exp + at, slots, held);
        }
    };
    const int warp = threadIdx.x >> 5, blocks = gridDim.x - 1;
    if (static_cast<int>(blockIdx.x) < blocks) {
        const long long items = static_cast<long long>(min(p.rows, __ldg(p.cu + p.R))) * p.parts;
        for (long long t = blockIdx.x * kWarps + warp; t < items; t += blocks * kWarps)
            do_row(static_cast<int>(t / p.parts), static_cast<int>(t % p.parts), -1);
    } else if (check_windows<kThreads>(p.cu, p.ctx, p.R, p.rows, tokens, p.dev_status)) {
        for (int i = 0; i < p.R; ++i) {
            const Window w = window_of(p.cu, p.ctx, i, p.rows, 0x7fffffff, tokens);
            for (int k = warp; k < w.n; k += kWarps)
                for (int part = 0; part < p.parts; ++part) do_row(w.row0 + k, part, i);
        }
    }
}

template <int D, bool INTER>
void (*kernel_of(int to))(const RotateParams) {
    return to == TO_ROWS ? rotate_kernel<D, INTER, TO_ROWS>
           : to == TO_CACHE ? rotate_kernel<D, INTER, TO_CACHE> : rotate_kernel<D, INTER, TO_CACHE_E4M3>;
}

}  // namespace

cudaError_t launch_rotate(const RotateParams& p, int D, bool interleaved, cudaStream_t s) {
    RotateParams q = p;
    const int vectors = p.H + (p.cached ? 2 : 1) * p.G;
    // few rows: a row's vectors go to several warps, down to one pass each
    const long long want = 16LL * num_sms() / std::max(p.rows, 1);
    q.parts = static_cast<int>(std::max<long long>(1, std::min<long long>(want, (vectors + 3) / 4)));
    const long long items = static_cast<long long>(p.rows) * q.parts;
    const int blocks = static_cast<int>(std::min<long long>((items + kWarps - 1) / kWarps, 8LL * num_sms()));
    const int to = !p.cached ? TO_ROWS : p.c.e4m3 ? TO_CACHE_E4M3 : TO_CACHE;
    auto k = D == 128 ? (interleaved ? kernel_of<128, true>(to) : kernel_of<128, false>(to))
                      : (interleaved ? kernel_of<64, true>(to) : kernel_of<64, false>(to));
    return launch_pdl(k, dim3(blocks + 1), dim3(kThreads), 0, s, q);
}

}  // namespace sdm
