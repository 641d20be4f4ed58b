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

// A warp takes a row's vectors (its query heads, key heads and, with a cache,
// value heads), or one of `parts` equal shares of them.  D / 8 lanes hold one
// vector, each lane two pieces of 4 elements such that a pair's two elements
// are one lane's: the same 4 angles serve every vector, and nothing but the
// sum of squares crosses lanes.
template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads) rotate_kernel(const RotateParams p) {
    constexpr int kLanes = D / 8;           // lanes per vector
    constexpr int kPer = 32 / kLanes;       // vectors per warp pass
    constexpr int kBatch = 4;               // passes whose loads are in flight together
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int sub = lane / kLanes, l = lane % kLanes;
    const int heads = p.H + p.G, vectors = heads + (p.cached ? p.G : 0);
    const long long tokens = p.cached ? table_tokens(p.c) : static_cast<long long>(kMaxTokens);
    // the lane's pieces of a rotated vector
    const int half = p.rot / 8;             // pieces of a half; lanes that rotate
    const bool turns = l < half;
    const int r0 = INTER ? 2 * l : turns ? l : 2 * half + 2 * (l - half);
    const int r1 = INTER ? 2 * l + 1 : turns ? l + half : r0 + 1;

    auto do_row = [&](int row, int part, int known) {
        const int v_from = static_cast<int>(static_cast<long long>(vectors) * part / p.parts);
        const int v_to = static_cast<int>(static_cast<long long>(vectors) * (part + 1) / p.parts);
        bool found = false, ok = false, held = false;
        size_t at = 0;
        float cs[4], sn[4];
        for (int v0 = v_from; v0 < v_to; v0 += kPer * kBatch) {
            uint2 x[kBatch][2];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const int vec = v0 + b * kPer + sub;
                const uint16_t* src = vec < p.H ? p.q + row * p.q_stride + static_cast<size_t>(vec) * D
                                      : vec < heads ? p.k + row * p.k_stride + static_cast<size_t>(vec - p.H) * D
                                                    : p.v + row * p.v_stride + static_cast<size_t>(vec - heads) * D;
                const bool plain = vec >= heads;   // values pass: contiguous pieces
                x[b][0] = x[b][1] = make_uint2(0, 0);
                if (vec < v_to) {
                    const uint2* s2 = reinterpret_cast<const uint2*>(src);
                    x[b][0] = s2[plain ? 2 * l : r0];   // not by the read-only path: the outputs may be the inputs
                    x[b][1] = s2[plain ? 2 * l + 1 : r1];
                }
            }
            if (!found) {
                found = true;
                const int i = known >= 0 ? known : warp_find_request(p.cu, p.R, row);
                const Window w = window_of(p.cu, p.ctx, i, p.rows, 0x7fffffff, tokens);
                if (row >= w.row0 && row < w.row0 + w.n) {
                    ok = true;
                    const int off = row - w.row0;
                    if (p.cached) {
                        const int pg = page_of(p.c, i, w.ctx + off);
                        held = pg >= 0;
                        if (held) at = pool_row(p.c, pg, w.ctx + off);
                        else if (lane == 0) set_status(p.dev_status, SDM_DEV_BAD_PAGE);
                    }
                    const long long first = p.start ? __ldg(p.start + i) : w.ctx;
                    const double pos = static_cast<double>(first + (p.row_pos ? __ldg(p.row_pos + row) : off));
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        cs[j] = 1.f;
                        sn[j] = 0.f;
                        if (turns) {
                            constexpr double kInv2Pi = 0.15915494309189533577;
                            const double t = pos * __ldg(p.freq + 4 * l + j) * kInv2Pi;
                            sincospif(2.0f * static_cast<float>(t - rint(t)), &sn[j], &cs[j]);
                        }
                    }
                }
            }
            if (!ok) break;
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const int vec = v0 + b * kPer + sub;
                uint32_t u[4] = {x[b][0].x, x[b][0].y, x[b][1].x, x[b][1].y};
                const bool is_q = vec < p.H, plain = vec >= heads;
                const float* weight = is_q ? p.q_weight : p.k_weight;
                float f[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = bf16_bits_to_float((u[j >> 1] >> (16 * (j & 1))) & 0xffffu);
                // all lanes of the warp take part in the sum, whatever their vector is
                if (p.q_weight || p.k_weight) {
                    float sum = 0.f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum = fmaf(f[j], f[j], sum);
#pragma unroll
                    for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    if (!plain && weight) {
                        const float inv = rsqrtf(sum * (1.0f / D) + p.eps);
                        const float4 w0 = __ldg(reinterpret_cast<const float4*>(weight) + r0);
                        const float4 w1 = __ldg(reinterpret_cast<const float4*>(weight) + r1);
                        f[0] *= inv * w0.x, f[1] *= inv * w0.y, f[2] *= inv * w0.z, f[3] *= inv * w0.w;
                        f[4] *= inv * w1.x, f[5] *= inv * w1.y, f[6] *= inv * w1.z, f[7] *= inv * w1.w;
                    }
                }
                if (!plain) {
                    if (turns) {
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
                const int o0 = plain ? 2 * l : r0, o1 = plain ? 2 * l + 1 : r1;
                if (is_q || !p.cached) {
                    uint16_t* dst = is_q ? p.q_out + row * p.q_out_stride + static_cast<size_t>(vec) * D
                                         : p.k_out + row * p.k_out_stride + static_cast<size_t>(vec - p.H) * D;
                    if (vec < v_to) {
                        reinterpret_cast<uint2*>(dst)[o0] = make_uint2(u[0], u[1]);
                        reinterpret_cast<uint2*>(dst)[o1] = make_uint2(u[2], u[3]);
                    }
                }
                if (!p.cached) continue;
                const int h = plain ? vec - heads : vec - p.H;
                const size_t r = at + (static_cast<size_t>(h) << p.c.page_shift);
                const bool put = held && !is_q && vec < v_to;
                if (!p.c.e4m3) {
                    if (put) {
                        uint2* dst = reinterpret_cast<uint2*>((plain ? p.c.v : p.c.k) + r * D * 2);
                        dst[o0] = make_uint2(u[0], u[1]);
                        dst[o1] = make_uint2(u[2], u[3]);
                    }
                } else {
                    const int e = e4m3_exponent<kLanes>(u);
                    const uint2 code = e4m3_codes(u, e);
                    if (put) {
                        uint32_t* dst = reinterpret_cast<uint32_t*>((plain ? p.c.v : p.c.k) + r * D);
                        dst[o0] = code.x;
                        dst[o1] = code.y;
                        if (l == 0) (plain ? p.c.v_exp : p.c.k_exp)[r] = static_cast<uint8_t>(e + 127);
                    }
                }
            }
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

}  // namespace

cudaError_t launch_rotate(const RotateParams& p, int D, bool interleaved, cudaStream_t s) {
    RotateParams q = p;
    const int vectors = p.H + (p.cached ? 2 : 1) * p.G;
    // few rows: a row's vectors go to several warps, down to one pass each
    const long long want = 16LL * num_sms() / std::max(p.rows, 1);
    q.parts = static_cast<int>(std::max<long long>(1, std::min<long long>(want, (vectors + 3) / 4)));
    const long long items = static_cast<long long>(p.rows) * q.parts;
    const int blocks = static_cast<int>(std::min<long long>((items + kWarps - 1) / kWarps, 8LL * num_sms()));
    auto k = D == 128 ? (interleaved ? rotate_kernel<128, true> : rotate_kernel<128, false>)
                      : (interleaved ? rotate_kernel<64, true> : rotate_kernel<64, false>);
    return launch_pdl(k, dim3(blocks + 1), dim3(kThreads), 0, s, q);
}

}  // namespace sdm
