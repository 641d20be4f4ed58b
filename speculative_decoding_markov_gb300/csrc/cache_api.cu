// cache_api.cu - the extern "C" entry points of the paged cache and the
// attention over it: argument validation and launches.  As everywhere in the
// library, work is enqueued on the caller's stream and nothing is allocated.
#include <algorithm>

#include "internal.h"

namespace {
using namespace sdm;

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// SDM_OK and the kernels' view of the cache, or what is wrong with it.
sdm_status view_of(const sdm_cache* c, CacheView* v) {
    if (!c || !c->k || !c->v || !c->table) return SDM_ERR_INVALID_ARG;
    if (c->dtype != SDM_BF16 && c->dtype != SDM_E4M3) return SDM_ERR_INVALID_ARG;
    if (c->n_pages <= 0 || c->kv_heads <= 0 || c->max_pages <= 0) return SDM_ERR_INVALID_ARG;
    const bool e4m3 = c->dtype == SDM_E4M3;
    if (e4m3 && (!c->k_exp || !c->v_exp)) return SDM_ERR_INVALID_ARG;
    if (c->head_dim != 64 && c->head_dim != 128) return SDM_ERR_UNSUPPORTED;
    if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128) return SDM_ERR_UNSUPPORTED;
    if (static_cast<long long>(c->n_pages) * c->kv_heads >= (1ll << 31) / c->page) return SDM_ERR_UNSUPPORTED;
    if (!aligned16(c->k) || !aligned16(c->v)) return SDM_ERR_UNSUPPORTED;
    if (e4m3 && (!aligned16(c->k_exp) || !aligned16(c->v_exp))) return SDM_ERR_UNSUPPORTED;
    v->k = static_cast<uint8_t*>(c->k);
    v->v = static_cast<uint8_t*>(c->v);
    v->k_exp = e4m3 ? c->k_exp : nullptr;
    v->v_exp = e4m3 ? c->v_exp : nullptr;
    v->table = c->table;
    v->e4m3 = e4m3;
    v->n_pages = c->n_pages;
    v->heads = c->kv_heads;
    v->page_shift = c->page == 16 ? 4 : c->page == 32 ? 5 : c->page == 64 ? 6 : 7;
    v->D = c->head_dim;
    v->max_pages = c->max_pages;
    return SDM_OK;
}

// Whether the grids' strides over rows and requests (below 65536) stay within 32 bits.
inline bool counts_ok(int R, int rows) { return R <= 0x7fff0000 && rows <= 0x7fff0000; }

// A row stride in elements: 16-byte rows that hold `width` elements.
inline bool stride_ok(int64_t stride, long long width) { return stride % 8 == 0 && stride >= width; }

}  // namespace

extern "C" {

sdm_status sdm_cache_write(const sdm_cache* cache, const uint16_t* k, const uint16_t* v, int64_t k_stride,
                           int64_t v_stride, const int32_t* cu_seqlens, const int32_t* ctx_len, int R, int rows,
                           int32_t* dev_status, void* stream) {
    CacheWriteParams p = {};
    if (!cu_seqlens || !ctx_len || R <= 0 || rows < 0) return SDM_ERR_INVALID_ARG;
    const sdm_status st = view_of(cache, &p.c);
    if (st != SDM_OK || rows == 0) return st;   // arrays without rows may have no address
    if (!k || !v) return SDM_ERR_INVALID_ARG;
    if (!counts_ok(R, rows)) return SDM_ERR_UNSUPPORTED;
    const long long width = static_cast<long long>(p.c.heads) * p.c.D;
    if (!stride_ok(k_stride, width) || !stride_ok(v_stride, width) || !aligned16(k) || !aligned16(v))
        return SDM_ERR_UNSUPPORTED;
    p.k = k;
    p.v = v;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.cu = cu_seqlens;
    p.ctx = ctx_len;
    p.R = R;
    p.rows = rows;
    p.dev_status = dev_status;
    return launch_cache_write(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SDM_OK : SDM_ERR_CUDA;
}

sdm_status sdm_cache_read(const sdm_cache* cache, const int32_t* cu_rows, const int32_t* first, int R, int rows,
                          uint16_t* k_out, uint16_t* v_out, int32_t* dev_status, void* stream) {
    CacheReadParams p = {};
    if (!cu_rows || R <= 0 || rows < 0) return SDM_ERR_INVALID_ARG;
    const sdm_status st = view_of(cache, &p.c);
    if (st != SDM_OK || rows == 0) return st;
    if (!k_out || !v_out) return SDM_ERR_INVALID_ARG;
    if (!counts_ok(R, rows) || !aligned16(k_out) || !aligned16(v_out)) return SDM_ERR_UNSUPPORTED;
    p.cu = cu_rows;
    p.first = first;
    p.k_out = k_out;
    p.v_out = v_out;
    p.R = R;
    p.rows = rows;
    p.dev_status = dev_status;
    return launch_cache_read(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SDM_OK : SDM_ERR_CUDA;
}

sdm_status sdm_cache_commit(const sdm_cache* cache, const int32_t* tok, const int32_t* parent,
                            const int32_t* n_nodes, const int32_t* out_tok, const int32_t* accept,
                            const int32_t* ctx_len, int R, int N, int B, int32_t* path, int32_t* length,
                            int32_t* dev_status, void* stream) {
    CacheCommitParams p = {};
    if (!tok || !parent || !n_nodes || !out_tok || !accept || !ctx_len || !path || R <= 0 || N < 0 || B <= 0)
        return SDM_ERR_INVALID_ARG;
    const sdm_status st = view_of(cache, &p.c);
    if (st != SDM_OK) return st;
    if (N >= kCommitMost || B > kCommitMost) return SDM_ERR_UNSUPPORTED;   // held in shared memory
    p.tok = tok;
    p.parent = parent;
    p.n_nodes = n_nodes;
    p.out_tok = out_tok;
    p.accept = accept;
    p.ctx = ctx_len;
    p.path = path;
    p.length = length;
    p.R = R;
    p.N = N;
    p.B = B;
    p.dev_status = dev_status;
    return launch_cache_commit(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SDM_OK : SDM_ERR_CUDA;
}

sdm_status sdm_attend(const sdm_cache* cache, const uint16_t* q, int64_t q_stride, const int32_t* cu_seqlens,
                      const int32_t* ctx_len, int R, int rows, int max_window, int H, float scale, int window,
                      int sinks, const int32_t* tree_mask, int tree_nodes, uint16_t* out, float* lse, void* ws,
                      size_t ws_bytes, int32_t* dev_status, void* stream) {
    AttendParams p = {};
    if (!cu_seqlens || !ctx_len || R <= 0 || rows < 0 || max_window < 0 || H <= 0) return SDM_ERR_INVALID_ARG;
    if (rows > 0 && (!q || !out || max_window == 0)) return SDM_ERR_INVALID_ARG;
    // the kernel works with scale * log2 e, which has to stay finite
    if (!(scale > 0.f) || scale > 2.0e38f || sinks < 0) return SDM_ERR_INVALID_ARG;
    if (tree_mask && tree_nodes < max_window) return SDM_ERR_INVALID_ARG;
    const sdm_status st = view_of(cache, &p.c);
    if (st != SDM_OK) return st;
    if (H % p.c.heads != 0) return SDM_ERR_INVALID_ARG;
    if (rows == 0) return SDM_OK;
    if (R > 16384 || !stride_ok(q_stride, static_cast<long long>(H) * p.c.D) || !aligned16(q) || !aligned16(out))
        return SDM_ERR_UNSUPPORTED;
    if (H / p.c.heads > 128) return SDM_ERR_UNSUPPORTED;   // a token's rows have to fit one tile
    // rows of one request and kv head are counted in 32 bits
    if (static_cast<long long>(max_window) * (H / p.c.heads) >= (1ll << 30)) return SDM_ERR_UNSUPPORTED;
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < attend_workspace(max_window, H, p.c.D, p.c.heads))
        return SDM_ERR_WORKSPACE;
    p.q = q;
    p.q_stride = q_stride;
    p.cu = cu_seqlens;
    p.ctx = ctx_len;
    p.R = R;
    p.rows = rows;
    p.max_window = max_window;
    p.H = H;
    p.group = H / p.c.heads;
    p.sub = 128 / p.group * p.group;
    p.scale = scale;
    p.window = std::max(window, 0);
    p.sinks = std::min(sinks, kMaxTokens);   // no cache holds more, and the kernel rounds it up to whole tiles
    p.tree = reinterpret_cast<const uint32_t*>(tree_mask);
    p.nodes = tree_mask ? tree_nodes : 0;
    p.words = (p.nodes + 31) / 32;
    p.out = out;
    p.lse = lse;
    p.dev_status = dev_status;
    return launch_attend(p, ws, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SDM_OK : SDM_ERR_CUDA;
}

}  // extern "C"
