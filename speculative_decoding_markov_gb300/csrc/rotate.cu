// rotate.cu - queries and keys normalised per head and rotated by their
// positions, the keys and values written into the paged cache on the way.
//
// Mathematics, per head vector x of D elements:
//     y = x rsqrt(mean(x^2) + eps) weight          (no weight: y = x)
//     (a, b) -> (a cos t - b sin t, b cos t + a sin t),  t = position freq_j
// for the pairs j < rot / 2: elements (j, j + rot / 2), or (2 j, 2 j + 1) if
// interleaved; elements from rot on pass.  Everything is fp32 and rounded to
// bf16 once, but the angle: at positions of 10^5 a fp32 product is off by
// 0.01 rad, so the turns position freq / 2 pi are reduced in fp64, and what the
// fp32 sine and cosine do not see of them is added to first order (without it
// results are off by 1e-7, and one in 20,000 is rounded the other way; 31 in a
// million with it).
//
// What bounds it (32 query heads on 8 kv heads of 128): a prompt of 8192 tokens
// into a bf16 cache 39.7 us, 5.1 TB/s, with half of the issue slots taken (e4m3:
// 52 us); 256 windows of 1 to 9 (28 heads on 4) into an e4m3 cache, read back,
// 14.6 us in a graph and one token 4.5 us, both a chain of dependent loads:
// offsets, table, rows.
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

__device__ __forceinline__ float2 mul2(float2 x, float2 y) {
    float2 r;
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmul.rn.f32x2 a, a, b;\n\t"
        "mov.b64 {%0, %1}, a;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y), "f"(z.x), "f"(z.y));
    return r;
}

// What __double2float_rz cuts off x (|x| < 1), times 2 pi: the last 29 bits, by
// integers, for fp64 instructions are few a clock (with two more of them an
// angle, a prompt of 8192 takes 41.3 us in place of 39.6).
__device__ __forceinline__ float rest_of(double x) {
    const int hi = __double2hiint(x);
    const int power = max(((hi >> 20) & 0x7ff) - 1023 - 52 + 127, 0);   // of the last bit
    const float unit = __int_as_float((power << 23) | (hi & static_cast<int>(0x80000000u)));
    return static_cast<float>(__double2loint(x) & 0x1fffffff) * (unit * 6.2831853f);
}

// One row's vectors first .. last - 1 of queries, keys or values (PLAIN): D / 8
// lanes a vector, kBatch passes of the warp loaded together.  (The next ones loaded
// while these are worked on: 44 us for a prompt of 8192 in place of 39, for the
// registers cost a third of the resident warps.)
template <int D, bool INTER, bool PLAIN, int TO, int kBatch>
__device__ __forceinline__ void section(const Lane& n, const uint16_t* src, int first, int last, const float* weight,
                                        float eps, const float (&cs)[4], const float (&sn)[4], uint8_t* dst,
                                        size_t head_bytes, uint8_t* exps, size_t head_rows, bool put) {
    constexpr int kLanes = D / 8, kPer = 32 / kLanes;
    const int p0 = PLAIN ? 2 * n.l : n.r0, p1 = PLAIN ? 2 * n.l + 1 : n.r1;
    // weight and rotation in one: (a, b) -> (a wa cos - b wb sin, b wb cos + a wa sin),
    // pair by pair, two pairs a register pair; 1 / norm comes after
    float2 ac[2], bs[2], bc[2], as[2];
    if constexpr (!PLAIN) {
        float w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = 1.f;
        if (weight) {
            const float4 a = __ldg(reinterpret_cast<const float4*>(weight) + p0);
            const float4 b = __ldg(reinterpret_cast<const float4*>(weight) + p1);
            w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float a0 = w[INTER ? 4 * j : 2 * j], a1 = w[INTER ? 4 * j + 2 : 2 * j + 1];
            const float b0 = w[INTER ? 4 * j + 1 : 2 * j + 4], b1 = w[INTER ? 4 * j + 3 : 2 * j + 5];
            ac[j] = make_float2(a0 * cs[2 * j], a1 * cs[2 * j + 1]);
            as[j] = make_float2(a0 * sn[2 * j], a1 * sn[2 * j + 1]);
            bc[j] = make_float2(b0 * cs[2 * j], b1 * cs[2 * j + 1]);
            bs[j] = make_float2(-b0 * sn[2 * j], -b1 * sn[2 * j + 1]);
        }
    }
    uint2 x[kBatch][2];
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
                for (int j = 0; j < 4; ++j) {
                    f[2 * j] = __uint_as_float(u[j] << 16);
                    f[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
                }
                float inv = 1.f;
                if (weight) {
                    float2 sq = mul2(make_float2(f[0], f[1]), make_float2(f[0], f[1]));
#pragma unroll
                    for (int j = 2; j < 8; j += 2) sq = fma2(make_float2(f[j], f[j + 1]), make_float2(f[j], f[j + 1]), sq);
                    float sum = sq.x + sq.y;
#pragma unroll
                    for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    inv = rsqrtf(fmaf(sum, 1.0f / D, eps));
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float& a0 = f[INTER ? 4 * j : 2 * j];
                    float& a1 = f[INTER ? 4 * j + 2 : 2 * j + 1];
                    float& b0 = f[INTER ? 4 * j + 1 : 2 * j + 4];
                    float& b1 = f[INTER ? 4 * j + 3 : 2 * j + 5];
                    const float2 a = make_float2(a0, a1), b = make_float2(b0, b1);
                    float2 x = mul2(a, ac[j]), y = mul2(b, bc[j]);
                    if (n.turns) {   // else an infinity would meet a sine of 0
                        x = fma2(b, bs[j], x);
                        y = fma2(a, as[j], y);
                    }
                    if (weight) {
                        x = mul2(x, make_float2(inv, inv));
                        y = mul2(y, make_float2(inv, inv));
                    }
                    a0 = x.x, a1 = x.y, b0 = y.x, b1 = y.y;
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
#pragma unroll 1
    for (int v0 = first; v0 < last; v0 += kStep) {
        load(v0, x);
        work(v0, x);
    }
}

// A warp takes a row, or one of `parts` equal shares of its vectors (query
// heads, key heads and, with a cache, value heads).
template <int D, bool INTER, int TO>
__global__ void __launch_bounds__(kThreads, 4) rotate_kernel(const RotateParams p) {
    constexpr int kLanes = D / 8, kBatch = 4;
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

    // `turn`: the rows' own outputs too, not only what goes into the cache
    auto do_row = [&](int row, int part, int known, bool turn) {
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
        // 4 angles a lane; the lanes of the pass's vectors that have the same share the work
        float cs[4], sn[4];
        constexpr int kPer = 32 / kLanes, kOwn = 4 / kPer;
#pragma unroll
        for (int j = 0; j < kOwn; ++j) {
            constexpr double kInv2Pi = 0.15915494309189533577;
            float c = 1.f, z = 0.f;
            if (n.turns) {
                const double t = pos * __ldg(p.freq + 4 * n.l + n.sub * kOwn + j) * kInv2Pi, part = t - rint(t);
                float s0, c0;
                sincospif(2.0f * __double2float_rz(part), &s0, &c0);
                const float rest = rest_of(part);
                c = fmaf(-s0, rest, c0);
                z = fmaf(c0, rest, s0);
            }
#pragma unroll
            for (int o = 0; o < kPer; ++o) {
                cs[o * kOwn + j] = __shfl_sync(0xffffffffu, c, n.l + o * kLanes);
                sn[o * kOwn + j] = __shfl_sync(0xffffffffu, z, n.l + o * kLanes);
            }
        }
        if (turn && v_from < p.H)
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
            do_row(static_cast<int>(t / p.parts), static_cast<int>(t % p.parts), -1, true);
    } else if (check_windows<kThreads>(p.cu, p.ctx, p.R, p.rows, tokens, p.dev_status)) {
        // The outputs may be the inputs, so that no row may be turned twice: rows
        // that the search finds are the other blocks', and of several windows
        // that hold one of the rest the first turns it.  (Every window's keys
        // and values go into its slots.)
        const int n_rows = min(p.rows, __ldg(p.cu + p.R));
        auto holds = [&](int i, int row) {
            const Window w = window_of(p.cu, p.ctx, i, p.rows, 0x7fffffff, tokens);
            return row >= w.row0 && row < w.row0 + w.n;
        };
        int reach = 0;   // no window before holds a row from here on
        for (int i = 0; i < p.R; ++i) {
            const Window w = window_of(p.cu, p.ctx, i, p.rows, 0x7fffffff, tokens);
            for (int k = warp; k < w.n; k += kWarps) {
                const int row = w.row0 + k;
                bool turn = true;
                if (row < n_rows) {
                    const int found = warp_find_request(p.cu, p.R, row);
                    if (found == i) continue;
                    turn = !holds(found, row);
                }
                for (int j = 0; turn && row < reach && j < i; j += 32)
                    turn = !__any_sync(0xffffffffu, j + lane < i && holds(j + lane, row));
                if (TO == TO_ROWS && !turn) continue;
                for (int part = 0; part < p.parts; ++part) do_row(row, part, i, turn);
            }
            reach = max(reach, w.row0 + w.n);
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
    // few rows: a row's vectors go to several warps, down to one pass each (8 or
    // 32 warps an SM wanted in place of 16: the same within 2 %)
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
