// paged.cuh - what the paged-cache kernels share: a packed row's request, a
// request's window, a token's slot, and the 8-bit format.
#pragma once
#include "device.cuh"
#include "internal.h"

namespace sdm {

// The largest i in [0, R) with cu[i] <= row, found by the whole warp (32
// probes a round).  cu need not be sound: the caller checks cu[i] <= row <
// cu[i + 1].
__device__ __forceinline__ int warp_find_request(const int32_t* cu, int R, int row) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = R;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) >> 5;
        const int at = lo + lane * step;
        const unsigned le = __ballot_sync(0xffffffffu, at < hi && __ldg(cu + at) <= row);
        const int last = le ? 31 - __clz(le) : 0;
        lo += last * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

// Request i's window: packed rows row0 .. row0 + n - 1 at tokens ctx, ctx +
// 1, ...; `bad` holds the SDM_DEV_* bits of what had to be cut.
struct Window {
    int row0, n, ctx, bad;
};

__device__ __forceinline__ Window window_of(const int32_t* cu, const int32_t* ctx_len, int i, int rows, int most,
                                            long long tokens) {
    Window w;
    w.row0 = __ldg(cu + i);
    const int end = __ldg(cu + i + 1);
    w.ctx = ctx_len ? __ldg(ctx_len + i) : 0;
    w.bad = 0;
    w.n = end - w.row0;
    if (w.row0 < 0 || end < w.row0 || end > rows) {
        w.n = 0;
        w.bad = SDM_DEV_BAD_WINDOW;
    }
    if (w.n > most) {
        w.n = most;
        w.bad |= SDM_DEV_BAD_WINDOW;
    }
    if (w.ctx < 0) {
        w.ctx = 0;
        w.bad |= SDM_DEV_BAD_WINDOW;
    }
    if (static_cast<long long>(w.ctx) + w.n > tokens) {
        w.ctx = static_cast<int>(min(static_cast<long long>(w.ctx), tokens));
        w.n = static_cast<int>(min(static_cast<long long>(w.n), tokens - w.ctx));
        w.bad |= SDM_DEV_BAD_PAGE;
    }
    return w;
}

__device__ __forceinline__ long long table_tokens(const CacheView& c) {
    const long long t = static_cast<long long>(c.max_pages) << c.page_shift;
    return t < kMaxTokens ? t : kMaxTokens;
}

// Page id of token `pos` of request i, or -1 (past the table or outside the pool).
__device__ __forceinline__ int page_of(const CacheView& c, int i, int pos) {
    const int col = pos >> c.page_shift;
    if (pos < 0 || col >= c.max_pages) return -1;
    const int pg = __ldg(c.table + static_cast<size_t>(i) * c.max_pages + col);
    return static_cast<unsigned>(pg) < static_cast<unsigned>(c.n_pages) ? pg : -1;
}

// Pool row (of head_dim elements) of head 0; head h is h << page_shift further.
__device__ __forceinline__ size_t pool_row(const CacheView& c, int pg, int pos) {
    return ((static_cast<size_t>(pg) * c.heads) << c.page_shift) + (pos & ((1 << c.page_shift) - 1));
}

// ---------------------------------------------------------------------------
// e4m3 and the power-of-two scales
// ---------------------------------------------------------------------------
constexpr int kExpLo = -110, kExpHi = 119;

__device__ __forceinline__ float pow2f(int e) {   // -126 <= e <= 127
    return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// The exponent byte of a stored scale: 0 and 255, which no write leaves and
// for which 2^(byte - 127) is no normal bf16, are read as 1 and 254.
__device__ __forceinline__ uint32_t scale_byte(uint32_t byte) { return min(max(byte, 1u), 254u); }
__device__ __forceinline__ float scale_of(uint32_t byte) { return pow2f(static_cast<int>(scale_byte(byte)) - 127); }

// Two codes (low byte first) as two fp16 values (every e4m3 value is one).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t codes) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(codes));
    return r;
}

__device__ __forceinline__ uint16_t f32x2_to_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t f32x2_to_bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float2 f16x2_to_f32x2(uint32_t h) {
    float2 r;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "r"(h));
    return r;
}

}  // namespace sdm
