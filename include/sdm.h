/*
 * sdm.h - C-ABI of the DSpark / PCTree speculative-decoding hot path on one
 * GB300 GPU (sm_103a).
 *
 * Library: libsdm.so (speculative_decoding_markov_gb300/libsdm.so).
 *
 * One decode cycle of semi-autoregressive speculative decoding is
 *   draft (Markov head, chain or PCTree)  ->  schedule (survival product and
 *   throughput-maximising prefix budget)  ->  pack (ragged front-pack into a
 *   captured tier)  ->  [target LLM forward: outside this library]  ->  verify.
 *
 * Sources, cited by page and section:
 *   [DSpark notes]  LayerX ML study-group notes (2026-06-30), summary of
 *                   "DSpark: Confidence-Scheduled Speculative Decoding with
 *                   Semi-Autoregressive Generation", sections 1-9.
 *   [PCTree]        Qiita article on PCTree (Parent-Conditioned Drafting Tree),
 *                   section on tree drafting with the Markov head.
 *   [SGLang]        "DSpark in SGLang" (winzheng.jp), sections on the SPS cost
 *                   table, ragged verify and the three verify modes.
 *
 * Conventions for every entry point:
 *   - Every pointer argument is a DEVICE pointer unless the comment says
 *     "host".  The caller owns every buffer; the library never allocates.
 *     Scratch memory is the caller's `ws` buffer of at least
 *     sdm_workspace_size(op, ...) bytes (256-byte aligned); calls, or graphs,
 *     that may run at the same time need one each.
 *   - Work is enqueued asynchronously on `stream` (a cudaStream_t passed as
 *     void*; NULL is the legacy default stream).  The return value reports
 *     host-side validation and launch errors only.
 *   - Conditions found on the device (out-of-range token ids, a verify window
 *     that does not fit, a bounded wait that ran out, a packed total above
 *     every tier) are OR-ed into *dev_status (device int32, SDM_DEV_* bits);
 *     the caller reads it after synchronising.  No kernel traps.
 *   - Layouts are row-major.  bf16 arrays are raw 16-bit patterns.
 *     L is [R, B, V]: L[i, d-1, :] is the backbone logit row of draft
 *     position d of request i.  U is [V, r], W is [r, V].
 *   - Constraints: V % 8 == 0, r % 64 == 0 and r <= 256, L/U/W/target base
 *     addresses 16-byte aligned.  Anything else returns SDM_ERR_UNSUPPORTED.
 *   - Randomness (sampling only) is Philox4x32-10 with key (seed mod 2^32,
 *     seed >> 32) and counter (0, request, stream << 16 | row,
 *     cycle mod 2^32); its word 0, w, gives u = (2 (w >> 9) + 1) 2^-24, one
 *     uniform per decision.  Streams: 0 draft, 1 accept test, 2 residual,
 *     3 bonus.
 *   - Ties: argmax and top-k prefer the lowest token id; the scheduler ranks
 *     (survival desc, request asc, position asc); PCTree prunes by (score
 *     desc, parent slot asc, child rank asc) and selects by (score desc,
 *     depth asc, creation order asc).
 *   - Calls are independent (no global state); results are deterministic.
 */
#ifndef SDM_H
#define SDM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    SDM_OK = 0,
    SDM_ERR_INVALID_ARG = 1,   /* null pointer, non-positive size, bad enum */
    SDM_ERR_UNSUPPORTED = 2,   /* shape or alignment outside the constraints */
    SDM_ERR_TIER_OVERFLOW = 3, /* strict tier mode: packed total above every tier (from sdm_status_of_device) */
    SDM_ERR_CUDA = 4,          /* a CUDA runtime or driver call failed */
    SDM_ERR_WORKSPACE = 5,     /* ws is NULL or smaller than required */
    SDM_ERR_DEVICE = 6,        /* a device-side input check failed (from sdm_status_of_device) */
    SDM_ERR_TIMEOUT = 7        /* a bounded device wait ran out (from sdm_status_of_device) */
} sdm_status;

/* SDM_E4M3 (8-bit floating point: sign, 4 exponent and 3 mantissa bits,
 * finite up to 448, one NaN) only as the element type of a paged cache. */
typedef enum { SDM_BF16 = 0, SDM_FP32 = 1, SDM_E4M3 = 2 } sdm_dtype;
typedef enum { SDM_GREEDY = 0, SDM_SAMPLE = 1 } sdm_decode;
typedef enum { SDM_STATIC = 0, SDM_COMPACT = 1, SDM_CAP_ACCEPT = 2 } sdm_vmode;

/* bits OR-ed into *dev_status */
enum {
    SDM_DEV_BAD_TOKEN = 1,        /* a token id outside [0, V) was read */
    SDM_DEV_TIER_UNCAPTURED = 2,  /* packed total above every tier: tier = total */
    SDM_DEV_TIMEOUT = 4,          /* a bounded pipeline wait ran out */
    SDM_DEV_BAD_WINDOW = 8,       /* budget or cu_seqlens window outside [0, gamma] */
    SDM_DEV_CAPACITY = 16,        /* packed rows would exceed the given capacity */
    SDM_DEV_BAD_CLASS = 32,       /* a request class id outside [0, n_class) */
    SDM_DEV_TIER_OVERFLOW = 64,   /* strict pack: packed total above every tier */
    SDM_DEV_BAD_PAGE = 128        /* paged cache: a page id outside the pool, or a token past the page table */
};

/* The status a caller reports for the device bits it read back after
 * synchronising: SDM_OK for 0 or SDM_DEV_TIER_UNCAPTURED alone (informational:
 * the caller runs that cycle uncaptured); else, by precedence,
 * SDM_ERR_TIMEOUT (SDM_DEV_TIMEOUT), SDM_ERR_TIER_OVERFLOW
 * (SDM_DEV_TIER_OVERFLOW), SDM_ERR_DEVICE (any other bit). */
sdm_status sdm_status_of_device(int32_t dev_status_bits);

/* Philox key material: key = seed, counter word 3 = cycle. */
typedef struct {
    uint64_t seed;
    uint64_t cycle;
} sdm_rng;

/* Operation ids for sdm_workspace_size. */
enum {
    SDM_OP_DRAFT_CHAIN = 0,
    SDM_OP_DRAFT_TREE = 1,
    SDM_OP_SCHEDULE = 2,
    SDM_OP_PACK = 3,
    SDM_OP_VERIFY = 4,
    SDM_OP_VERIFY_TREE = 5,
    SDM_OP_TV_LABEL = 6,
    SDM_OP_DRAFT_CHAIN_RNN = 7,
    SDM_OP_ATTEND = 8,
    SDM_OP_ATTEND_WEIGHT = 9,
    SDM_OP_CACHE_EVICT = 10
};

/* Bytes of scratch the operation needs for these sizes (0 if none).  Pass the
 * same sizes as the call; unused sizes may be 0.  For SDM_OP_VERIFY and
 * SDM_OP_TV_LABEL pass the packed row capacity as P. */
size_t sdm_workspace_size(int op, int R, int B, int V, int r, int P, int k, int N);

/*
 * markov_prepare: tables derived once from the Markov head (U, W), for the
 * greedy chain (no counterpart on the pages; a weight-preparation step, like
 * packing a weight matrix at load time).  Fills `prepared` (device, at least
 * sdm_markov_prepared_size(V, r) bytes, 256-byte aligned) with, in order,
 * each array starting on a 256-byte boundary:
 *   W^T [V, r] bf16;
 *   c [V] fp32: c(y) bounds |U[y] . W[:, v]| over every v, for the exact
 *     product and for any fp32 evaluation of it:
 *       c(y) = A(y) (1 + 2^-10) + 4 r 2^-24 |U[y]|_2 max_v |W[:, v]|_2 + 2^-20
 *     rounded up, A(y) = max_v |U[y] . W[:, v]| accumulated in fp32 by the
 *     tensor cores (one V x V x r product, about 12 TFLOP at V = 151,936,
 *     r = 256; nothing of it is stored);
 *   |U[v]|_2 [V] fp32 (fp64 accumulation, rounded up); A [V] (scratch);
 *   c_max = max_y c(y), max_v |W[:, v]|_2, max_v |U[v]|_2 (fp32 each).
 * A pipeline wait that runs out sets SDM_DEV_TIMEOUT in *dev_status (may be
 * NULL).  Enqueued on `stream`; valid until U or W change.
 */
size_t sdm_markov_prepared_size(int V, int r);
sdm_status sdm_markov_prepare(const uint16_t* U, const uint16_t* W, int V, int r, void* prepared,
                              size_t prepared_bytes, int32_t* dev_status, void* stream);

/*
 * draft_chain: the Markov-head sequential stage ([DSpark notes] sec. 4,
 * "Sequential stage" and "Markov head"; [PCTree] z_d = L_d + Markov(y_{d-1})).
 * For d = 1..B, with y_0 = anchor:
 *     z_d = fp32(L[i, d-1, :]) + U[y_{d-1}] . W          (fp32)
 *     greedy:  y_d = argmax_v z_d[v]
 *     sample:  y_d ~ softmax(z_d / T) by the inverse CDF in vocabulary
 *              order: the smallest v with sum_{j<=v} exp(z_d[j]/T) > u S,
 *              S the sum over all j, u = the uniform of (stream 0, row d);
 *              lse[i, d-1] = log sum_v exp(z_d[v]/T);
 *              logq[i, d-1] = z_d[y_d]/T - lse[i, d-1].
 * In:  L [R, B, V] (dtL), U [V, r] bf16, W [r, V] bf16, anchor [R] int32;
 *      prepared: NULL, or the tables sdm_markov_prepare built from U and W.
 * Out: tokens [R, B] int32; logq, lse [R, B] fp32 (sample only; may be NULL
 *      when greedy).
 * Sampling (and greedy without prepared tables): the product U[y] . W runs on
 * the tcgen05 tensor cores (bf16 in, fp32 accumulate in TMEM) and the +L /
 * argmax (greedy) or per-16-column (max, sum of exp) records (sampling) are
 * fused into its epilogue; z is never written to memory.  A sampled step
 * then walks the records of each request to the block holding u S and
 * recomputes that block's 16 logits to find the id (V <= 524288, else
 * SDM_ERR_UNSUPPORTED).
 * Greedy with prepared tables: since |U[y] . W[:, v]| <= c(y) for every v,
 * only ids with L[v] >= max L - 2 c(y) can win.  One HBM-bound pass over all
 * of L lists those ids for every (request, step) with the worst case c_max,
 * then one CTA per request stages the listed rows of W^T and U in shared
 * memory and walks the B steps, scoring exactly the ids that the previous
 * token's c(y) leaves.  L is read once and the result is the same argmax bit
 * for bit.  Needs B <= 64, V <= 64 * 16384 (bf16 L) or 64 * 8192 (fp32 L) and
 * R * B * ceil(V / 16384 or 8192) <= 2^30, else SDM_ERR_UNSUPPORTED.
 */
sdm_status sdm_draft_chain(const void* L, sdm_dtype dtL, const uint16_t* U, const uint16_t* W,
                           const void* prepared, const int32_t* anchor, int R, int B, int V, int r,
                           sdm_decode decode, float temperature, sdm_rng rng,
                           int32_t* tokens, float* logq, float* lse,
                           void* ws, size_t ws_bytes, int32_t* dev_status, void* stream);

/*
 * draft_chain_packed: the greedy chain of sdm_draft_chain with prepared
 * tables, writing its drafts also into the ragged verify layout (the pack of
 * [SGLang] "ragged verify" without a pass of its own after the draft).  The
 * layout is sdm_pack_ragged's with draft = NULL (cu_seqlens, the tier, the
 * row maps and the anchors, made from the budgets alone, e.g. on a second
 * stream while this draft runs); this call fills rows cu[i] + 1 .. cu[i] +
 * n_i of packed_tok with y_1 .. y_{n_i}, n_i = cu[i+1] - cu[i] - 1, so that
 * packed_tok ends as sdm_pack_ragged with the drafts would leave it.
 * layout_ready (a cudaEvent_t, may be NULL): recorded after the layout's
 * producer; the scan of L starts at once, the pass that writes the drafts
 * waits for the event on `stream`.  NULL: the layout is ordered before this
 * call on `stream`.
 * In/out as sdm_draft_chain (prepared required); cu_seqlens [R+1],
 * packed_tok [capacity] (device).  A window longer than B sets
 * SDM_DEV_BAD_WINDOW (cut to B); rows past capacity SDM_DEV_CAPACITY.
 */
sdm_status sdm_draft_chain_packed(const void* L, sdm_dtype dtL, const uint16_t* U, const uint16_t* W,
                                  const void* prepared, const int32_t* anchor, int R, int B, int V, int r,
                                  const int32_t* cu_seqlens, int32_t* packed_tok, int capacity, void* layout_ready,
                                  int32_t* tokens, void* ws, size_t ws_bytes, int32_t* dev_status, void* stream);

/*
 * draft_chain_front: the greedy chain draft together with the budget
 * scheduler and the ragged layout of its windows, in one call whose outputs
 * equal, bit for bit, those of
 *     sdm_schedule_budget(conf, R, B, cost, survival, budget, expected,
 *                         total_tokens)
 *     sdm_pack_ragged(anchor, NULL, use_budget ? budget : NULL, R, B, tiers,
 *                     n_tiers, strict, cu_seqlens, packed_tok, packed_req,
 *                     packed_pos, capacity, tier)
 *     sdm_draft_chain_packed(L, ..., prepared, anchor, R, B, V, r,
 *                            cu_seqlens, packed_tok, capacity, NULL, tokens)
 * ([DSpark notes] sec. 4, 5.1-5.2; [SGLang] "ragged verify").  The scheduler
 * and the layout need only the confidences, so they run in one extra CTA of
 * the draft's first (vocabulary-streaming) launch, beside its other CTAs,
 * and the pick writes the drafts into the layout; nothing runs on a second
 * stream.  It pays when the scan fills every SM (a side-stream scheduler
 * then waits for the scan to drain: 67.4 against 70.5 us per decode cycle
 * of 64 requests, B 7, V 151936); on a scan of a few CTAs the scheduler's
 * CTA is the longer path, and the three calls with the scheduler on a second
 * stream are faster.  Requires the prepared tables and R * B <= 8192 with the
 * scheduler's shared memory (about 16 (R B) bytes rounded up) within 48 KB,
 * else SDM_ERR_UNSUPPORTED (use the three calls).  Arguments as in those
 * calls; use_budget 1 packs budget[i] drafts per request (compact), 0 all B
 * (static); the tier's host copy is not offered.  Workspace: as
 * SDM_OP_DRAFT_CHAIN.
 */
sdm_status sdm_draft_chain_front(const void* L, sdm_dtype dtL, const uint16_t* U, const uint16_t* W,
                                 const void* prepared, const int32_t* anchor, int R, int B, int V, int r,
                                 const float* conf, const double* cost, int use_budget, const int32_t* tiers,
                                 int n_tiers, int strict, float* survival, int32_t* budget, double* expected,
                                 int32_t* total_tokens, int32_t* cu_seqlens, int32_t* packed_tok, int32_t* packed_req,
                                 int32_t* packed_pos, int capacity, int32_t* tier, int32_t* tokens, void* ws,
                                 size_t ws_bytes, int32_t* dev_status, void* stream);

/*
 * draft_chain_rnn: the chain draft with the RNN sequential head ([DSpark
 * notes] sec. 4, "RNN head": a memo that carries the whole draft so far,
 * updated once per step from the previous memo, the previous word and the
 * current backbone state; the page's formula is not legible, the reading
 * taken is)
 *     m_0 = 0,  m_d = tanh(A m_{d-1} + U[y_{d-1}] + x_d)
 *     z_d = L_d + bf16(m_d) . W
 * then y_d as in draft_chain (greedy argmax, or the inverse-CDF draw of
 * softmax(z_d / T) with the same random stream).  With A = 0 and x = 0 this
 * is the Markov head on the table bf16(tanh(U)).
 * In:  L [R, B, V] (dtL), U [V, r], W [r, V], A [r, r] (row j = output j),
 *      X [R, B, r] (x_d: the backbone state at position d projected to r),
 *      all bf16 but L; anchor [R].  Shapes and alignment as draft_chain.
 * Out: tokens [R, B]; logq, lse [R, B] fp32 (sampling; may be NULL);
 *      memo [R, B, r] fp32 = m_d per position (may be NULL).  The memo is
 *      formed in fp32 (tanhf); the projection on the tensor cores with fp32
 *      accumulation.
 * ws:  sdm_workspace_size(SDM_OP_DRAFT_CHAIN_RNN, R, B, V, r, 0, 0, 0).
 * Device checks as draft_chain (a token id outside [0, V) sets
 * SDM_DEV_BAD_TOKEN and is read as 0).
 */
sdm_status sdm_draft_chain_rnn(const void* L, sdm_dtype dtL, const uint16_t* U, const uint16_t* W, const uint16_t* A,
                               const uint16_t* X, const int32_t* anchor, int R, int B, int V, int r, sdm_decode decode,
                               float temperature, sdm_rng rng, int32_t* tokens, float* logq, float* lse, float* memo,
                               void* ws, size_t ws_bytes, int32_t* dev_status, void* stream);

/*
 * draft_tree: PCTree drafting ([PCTree]: per parent p, z_d(p) = L_d +
 * Markov(p) for every frontier parent in one batched Markov call; local top-k
 * per parent; path score s(c) = s(p) + log pi(v | p); top-P prune per level;
 * global top-N selection within the verify budget; the tree is verified in one
 * target forward with a tree-causal mask ([DSpark notes] JetSpec note: a node
 * attends to its ancestors only)).
 * Level 1 expands the root (token anchor[i], score 0); level d expands the
 * <= P nodes kept at level d-1.  Scores use T = 1 and are fp32.
 * Out (per request, N+1 slots; slot 0 = root, then the selected nodes in
 * rank order so parent[c] < c; unused slots hold -1 / 0):
 *   tok, parent, depth [R, N+1] int32; score [R, N+1] fp32;
 *   mask [R, N+1, ceil((N+1)/32)] uint32, bit j of row c set iff slot j is c
 *   or an ancestor of c; n_nodes [R] int32 (root included).
 * prepared: NULL, or the tables sdm_markov_prepare built from U and W.
 * With prepared tables: since |U[y] . W[:, v]| <= c(y) for every v, the top
 * k ids of parent y have L[v] >= L_(k) - 2 c(y), L_(k) the k-th largest
 * backbone logit of the row.  One HBM-bound pass over L lists, per 32 KB
 * chunk of every (request, level) row, the ids with L >= theta - 2 c_max
 * (theta a lower bound on the chunk's k-th largest value); each level then
 * runs the tcgen05 GEMM for every frontier row with only an online
 * log-sum-exp in its epilogue, and one CTA per request scores the listed ids
 * each parent can need exactly (z = L + U[y] . W^T[v]), takes each parent's
 * top k, the children's scores and the prune.  A row whose lists overflow
 * takes the exact top k over the whole vocabulary instead (slow).  Needs
 * V <= 64 * 16384 (bf16 L) or 64 * 8192 (fp32 L), R B ceil(V / 16384 or
 * 8192) <= 2^30.
 * Without: each level runs the tcgen05 GEMM for every frontier row with
 * per-16-column (max, sum of exp) records in its epilogue; the row's top-k
 * ids lie in the k blocks with the largest maxima, so one CTA per row ranks
 * the records, recomputes the logits of its 2k best blocks and ranks those.
 * Both give the same tree.
 * Constraints: 1 <= k <= 8, 1 <= P, P*k <= 64, 128 % P == 0, N <= P*B,
 * P*B + 1 <= 8192, V <= 524288 (else SDM_ERR_UNSUPPORTED).
 */
sdm_status sdm_draft_tree(const void* L, sdm_dtype dtL, const uint16_t* U, const uint16_t* W, const void* prepared,
                          const int32_t* anchor, int R, int B, int V, int r, int k, int P, int N,
                          int32_t* tok, int32_t* parent, int32_t* depth, float* score,
                          uint32_t* mask, int32_t* n_nodes,
                          void* ws, size_t ws_bytes, int32_t* dev_status, void* stream);

/*
 * schedule_budget: confidence survival and the hardware-aware prefix budget
 * ([DSpark notes] sec. 5.1 and 5.2; [SGLang] "SPS cost table").
 *   S[i, k] = S[i, k-1] * c[i, k]  (fp32, k = 1..gamma, S[i, 0] = 1)
 *   Survivals >= 2^-18 are ranked (S desc, request asc, position asc); with
 *   E(m) = R + sum of the top m and N(m) = R + m, the greedy adds the next
 *   survival while E(m+1)/cost[N(m+1)] > E(m)/cost[N(m)] and stops at the
 *   first that does not improve it.  budget[i] = request i's count in the
 *   top m*.  Sums are exact in fp64.
 * In:  conf [R, gamma] fp32 (post-sigmoid), cost [R*(gamma+1)+1] fp64 (step
 *      cost by total verify tokens).
 * Out: survival [R, gamma] fp32, budget [R] int32, expected [1] fp64 (E(m*)),
 *      total_tokens [1] int32 (N(m*)).
 * Constraint: R * gamma <= 8192.
 */
sdm_status sdm_schedule_budget(const float* conf, int R, int gamma, const double* cost,
                               float* survival, int32_t* budget, double* expected,
                               int32_t* total_tokens, void* ws, size_t ws_bytes,
                               int32_t* dev_status, void* stream);

/*
 * schedule_dynamic: the production scheduler ([DSpark notes] sec. 9.2,
 * "scheduler adaptation on real hardware").  The step's batch capacity must
 * be known before the step's own confidences are, so it comes from the
 * confidences of two steps before; the step's candidates are still ranked by
 * their own survivals (dynamic top-K); and because the capacity no longer
 * depends on this step's tokens, the search over the cost table is global,
 * which crosses the steps of a tiered table that an early stop would not.
 *   S'[i, k], S[i, k]: the survival products of conf_stale and conf (fp32,
 *   left to right), ranked as in schedule_budget (S desc, request asc,
 *   position asc; values below 2^-18 are left out).
 *   K = the m in 0 .. (ranked S') maximising E'(m) / cost[R + m], E'(m) =
 *   R + sum of the top m of S' (exact fp64), the smallest m on ties.
 *   budget[i] = request i's count in the top min(K, ranked S) of S.
 * In:  conf, conf_stale [R, gamma] fp32 (post-sigmoid), cost
 *      [R*(gamma+1)+1] fp64, every entry > 0 (it may step with the tier).
 * Out: survival [R, gamma] fp32 (of conf), budget [R] int32, expected [1]
 *      fp64 (R + the selected survivals), total_tokens [1] int32
 *      (R + min(K, ranked S)), capacity [1] int32 (K).
 * Constraint: R * gamma <= 8192.
 */
sdm_status sdm_schedule_dynamic(const float* conf, const float* conf_stale, int R, int gamma,
                                const double* cost, float* survival, int32_t* budget,
                                double* expected, int32_t* total_tokens, int32_t* capacity,
                                int32_t* dev_status, void* stream);

/*
 * pack_ragged: ragged front-pack of the verify windows ([SGLang] "ragged
 * verify": windows are front-packed into a compact cu_seqlens buffer whose
 * total is rounded up to the nearest captured tier).
 *   n_i = budget[i] (budget == NULL: n_i = gamma, the static block)
 *   cu_seqlens[0] = 0, cu_seqlens[i+1] = cu_seqlens[i] + n_i + 1
 *   rows cu[i] .. cu[i] + n_i hold y_0 (anchor), y_1 .. y_{n_i}, with
 *   packed_req = i and packed_pos = 0..n_i; rows total .. capacity-1 hold -1.
 *   tier = smallest tiers[q] >= total; above every tier: tier = total and
 *   SDM_DEV_TIER_UNCAPTURED is set (the caller runs uncaptured), or, with
 *   strict != 0, SDM_DEV_TIER_OVERFLOW instead (a caller that only runs
 *   captured tiers maps it to SDM_ERR_TIER_OVERFLOW with
 *   sdm_status_of_device; the rows are packed the same way).
 * In:  anchor [R], draft [R, gamma] or NULL (the layout alone: every draft
 *      row holds -1, for sdm_draft_chain_packed to fill), budget [R] or
 *      NULL, tiers [n_tiers] int32 (device), strict (0 or 1).
 * Out: cu_seqlens [R+1], packed_tok/req/pos [capacity], tier [1] (device);
 *      tier_host (host, may be NULL): if non-NULL it must be pinned host
 *      memory and receives the tier by an async copy on `stream`.
 * capacity >= max(max tier, R*(gamma+1)) guarantees every row fits; rows past
 * capacity are dropped and SDM_DEV_CAPACITY is set.
 */
sdm_status sdm_pack_ragged(const int32_t* anchor, const int32_t* draft, const int32_t* budget,
                           int R, int gamma, const int32_t* tiers, int n_tiers, int strict,
                           int32_t* cu_seqlens, int32_t* packed_tok, int32_t* packed_req,
                           int32_t* packed_pos, int capacity, int32_t* tier, int32_t* tier_host,
                           int32_t* dev_status, void* stream);

/*
 * verify: fused verification over the packed target logits ([DSpark notes]
 * sec. 1: left-to-right acceptance, discard after the first rejection, one
 * bonus token; [SGLang] "three verify modes").
 * Window of request i: w_i = cu[i+1] - cu[i] - 1 drafts, target rows
 * cu[i] .. cu[i] + w_i; row p is the target's prediction after y_p.
 *   greedy: t_p = argmax target row p; A = first p < w_i with y_{p+1} != t_p,
 *           else w_i; commit a = A drafts and t_a.
 *   sample: accept y_{p+1} iff u(stream 1, row p) < p_p(y)/q_p(y), with
 *           p = softmax(target row / T) and q_p(y) = exp(logq[i, p]); at the
 *           first rejection p = a, sample from max(0, p_a - q_a) where q_a is
 *           recomputed from L, U, W and lse_q (stream 2, row a); if all
 *           committed drafts pass, the bonus is drawn from p at row a
 *           (stream 3).  Every draw is the inverse CDF in vocabulary order
 *           with one uniform (word 0 of the Philox block of its stream and
 *           row; the row of a draft is d, of an accept test, residual or
 *           bonus the window position).  Sampling needs V <= 524288 (else
 *           SDM_ERR_UNSUPPORTED).
 *   modes: STATIC (w_i = gamma, commit A), COMPACT (w_i = budget, commit A),
 *          CAP_ACCEPT (w_i = gamma verified, commit a = min(A, budget[i]):
 *          the same output as compact; ceiling = A).
 * In:  target [rows, V] (dtT), cu_seqlens [R+1], anchor [R], draft [R, gamma];
 *      budget [R] (CAP_ACCEPT only); logq, lse_q [R, gamma] fp32, L [R, gamma,
 *      V], U, W, r (SAMPLE only, else may be NULL/0).  row_capacity = rows
 *      allocated in target (an upper bound on cu[R]).
 * Out: accept [R], ceiling [R] (may be NULL), out_tok [R, gamma+1] (-1
 *      padded), n_out [R] = accept + 1.
 * Only rows below min(cu[R], row_capacity) are read.  A request without
 * rows (cu[i+1] <= cu[i]) or whose rows end past cu[R] (a non-monotone
 * cu_seqlens) sets SDM_DEV_BAD_WINDOW, one whose rows run past row_capacity
 * sets SDM_DEV_CAPACITY; such a request commits one token (0) with accept 0
 * (greedy and sample).  A window longer than gamma is flagged
 * (SDM_DEV_BAD_WINDOW) and cut to gamma.
 */
sdm_status sdm_verify(sdm_vmode mode, sdm_decode decode, float temperature, sdm_rng rng,
                      const void* target, sdm_dtype dtT, int row_capacity, const int32_t* cu_seqlens,
                      const int32_t* anchor, const int32_t* draft, const int32_t* budget,
                      const float* logq, const float* lse_q,
                      const void* L, sdm_dtype dtL, const uint16_t* U, const uint16_t* W, int r,
                      int R, int gamma, int V,
                      int32_t* accept, int32_t* ceiling, int32_t* out_tok, int32_t* n_out,
                      void* ws, size_t ws_bytes, int32_t* dev_status, void* stream);

/*
 * verify_tree: greedy verification of a drafted tree in one target forward
 * ([PCTree]; greedy only).  Walk from the root: t = argmax of the current
 * slot's target row; move to the child whose token is t; stop when none is.
 * accept = depth reached; out_tok = accepted tokens then t (bonus).
 * In:  target [R, N+1, V] (dtT; slot c's row predicts c's child), tok, parent
 *      [R, N+1], n_nodes [R].
 * Out: accept [R], out_tok [R, B+1] (-1 padded), n_out [R].
 * When several children carry t, the lowest slot is taken.  N < 16384, else
 * SDM_ERR_UNSUPPORTED.
 */
sdm_status sdm_verify_tree(const void* target, sdm_dtype dtT, const int32_t* tok,
                           const int32_t* parent, const int32_t* n_nodes, int R, int N, int B, int V,
                           int32_t* accept, int32_t* out_tok, int32_t* n_out,
                           void* ws, size_t ws_bytes, int32_t* dev_status, void* stream);

/*
 * verify_greedy_static: greedy verification (as sdm_verify with SDM_GREEDY)
 * that allocates nothing and takes no workspace.  The pages have no
 * counterpart; this entry point exists for callers that cannot hand the
 * library scratch memory: a server that reserved all device memory up front,
 * a framework whose allocator must account for every byte, or a latency-bound
 * loop that cannot afford the device synchronisation of cudaMalloc/cudaFree.
 * Scratch: a fixed 1 MiB array in the library's own device memory (every GPU
 * that loads libsdm.so holds it until the process exits); row_capacity *
 * ceil(V / 16384) (bf16 target) or row_capacity * ceil(V / 8192) (fp32) must
 * be <= 131072, else SDM_ERR_WORKSPACE and nothing is launched.
 * The first call on a device looks the array's device address up (once per
 * device, with that device current, and again if the device's context has
 * changed since, e.g. after a device reset); make that first call before any
 * stream capture.  All calls share the one array and each call rewrites every
 * partial it reads (rows below min(cu[R], row_capacity); a window past them is
 * flagged as in sdm_verify), so nothing carries over between calls, but calls
 * that overlap on the GPU (concurrent streams) race on it: serialise them.
 * Arguments and outputs are those of sdm_verify.
 */
sdm_status sdm_verify_greedy_static(sdm_vmode mode, const void* target, sdm_dtype dtT, int row_capacity,
                                    const int32_t* cu_seqlens, const int32_t* draft, const int32_t* budget,
                                    int R, int gamma, int V, int32_t* accept, int32_t* ceiling,
                                    int32_t* out_tok, int32_t* n_out, int32_t* dev_status, void* stream);

/*
 * check_timeout_path: exercises the device-side timeout path on purpose (no
 * counterpart on the pages; a failure-detection check).  Every pipeline wait
 * of the tensor-core kernels is bounded by a wall-clock limit (2 s in normal
 * calls); when one runs out the kernel ORs SDM_DEV_TIMEOUT into *dev_status,
 * waits (bounded) for the copies and tensor-core work it has in flight, frees
 * its tensor memory and returns, so the context stays usable.  This call
 * launches the greedy chain's Markov GEMM for step 1 on the given inputs with
 * its loads withheld and every wait limited to wait_ns (1 us .. 1 s), so
 * every wait runs out: afterwards *dev_status holds SDM_DEV_TIMEOUT and
 * later calls on the stream run normally.  Nothing but the keys in ws is
 * written.
 * In:  as sdm_draft_chain (dense path); ws at least
 *      sdm_workspace_size(SDM_OP_DRAFT_CHAIN, R, B, V, r, 0, 0, 0) bytes;
 *      dev_status must not be NULL.
 */
sdm_status sdm_check_timeout_path(const void* L, sdm_dtype dtL, const uint16_t* U, const uint16_t* W,
                                  const int32_t* anchor, int R, int B, int V, int r, unsigned long long wait_ns,
                                  void* ws, size_t ws_bytes, int32_t* dev_status, void* stream);

/* Human-readable name of a status code (static string). */
const char* sdm_status_str(sdm_status status);

/* Library version, major * 10000 + minor * 100 + patch. */
int sdm_version(void);

/*
 * schedule_threshold: the conventional fixed-threshold verify length
 * ([DSpark notes] sec. 5.2: a fixed threshold on the confidences decides how
 * many drafts are verified; sec. 8.3, Fig. 5).  budget[i] = the longest
 * prefix n such that conf[i, d] >= tau for every d < n (fp32 comparison; a
 * NaN confidence ends the prefix); total_tokens = R + sum_i budget[i] (every
 * request sends its root token).
 * In:  conf [R, gamma] fp32 (device), tau.  R gamma <= 2^30.
 * Out: budget [R] int32, total_tokens [1] int32 (device).
 */
sdm_status sdm_schedule_threshold(const float* conf, int R, int gamma, float tau, int32_t* budget,
                                  int32_t* total_tokens, int32_t* dev_status, void* stream);

/*
 * threshold_sweep: the fixed-threshold rule at K thresholds at once
 * ([DSpark notes] sec. 8.3, Fig. 5: threshold 0 verifies the whole block).
 * With n_i(tau) as in schedule_threshold, for threshold k:
 *   drafts[k]   = sum_i n_i(tau_k)                     drafts verified
 *   accepted[k] = sum_i min(ceiling[i], n_i(tau_k))    drafts accepted, given
 *                 the acceptance count of the whole block (sdm_verify's
 *                 ceiling in CAP_ACCEPT or STATIC mode); -1 if ceiling NULL
 *   expected[k] = sum_i sum_{d <= n_i} S_{i,d}         expected accepted drafts,
 *                 S the fp32 running products of conf ([DSpark notes] sec.
 *                 5.1), summed exactly: each S >= 2^-24 as an integer count
 *                 of 2^-48, smaller survivals counted 0.
 * In:  conf [R, gamma] fp32, ceiling [R] int32 or NULL, taus [K] fp32
 *      (device).  R gamma <= 32768 (the exact sum stays below 2^63), K <= 65535.
 * Out: drafts, accepted [K] int32, expected [K] fp64 (device).
 */
sdm_status sdm_threshold_sweep(const float* conf, const int32_t* ceiling, int R, int gamma, const float* taus, int K,
                               int32_t* drafts, int32_t* accepted, double* expected, int32_t* dev_status,
                               void* stream);

/*
 * tv_label: the confidence head's soft label for every verified draft position
 * ([DSpark notes] sec. 5.1: the label is the single-token acceptance rate,
 * fixed by the total-variation distance between the draft and target
 * distributions):
 *     label[i, p] = sum_v min(q_v, p_v) = 1 - TV(q, p)         for p < w_i
 * with q = softmax((L[i, p] + U[y_p] . W) / T) the draft's distribution at
 * position p+1 (y_0 = anchor[i], y_p = draft[i, p-1]) and p = softmax(target
 * row cu[i] + p / T); w_i = cu[i+1] - cu[i] - 1.  label[i, p] = -1 for
 * p >= w_i.
 * In:  target [row_capacity, V] (dtT, the packed verify rows), cu_seqlens
 *      [R+1], anchor [R], draft [R, gamma]; lse_q [R, gamma] fp32 = the
 *      draft's log-sum-exp of (L + Markov) / T, as sampling drafts return it,
 *      or NULL: computed here by one more pass over L; L [R, gamma, V] (dtL),
 *      U [V, r], W [r, V] bf16, r in {64, 128, 192, 256}; temperature > 0 (1
 *      for greedy drafts).  target, L, U, W 16-byte aligned; V % 8 == 0;
 *      R gamma <= 2^22.
 * Out: label [R, gamma] fp32 (device).  Arithmetic in fp32 (exp, sums over
 *      16-column blocks, then over the vocabulary splits in a fixed order).
 * ws:  sdm_workspace_size(SDM_OP_TV_LABEL, R, gamma, V, r, row_capacity, 0, 0).
 * Device checks (OR-ed into *dev_status, the row keeps label -1): windows
 * outside [0, gamma] SDM_DEV_BAD_WINDOW, target rows past row_capacity
 * SDM_DEV_CAPACITY, previous tokens outside [0, V) SDM_DEV_BAD_TOKEN.
 */
sdm_status sdm_tv_label(float temperature, const void* target, sdm_dtype dtT, int row_capacity,
                        const int32_t* cu_seqlens, const int32_t* anchor, const int32_t* draft, const float* lse_q,
                        const void* L, sdm_dtype dtL, const uint16_t* U, const uint16_t* W, int r, int R, int gamma,
                        int V, float* label, void* ws, size_t ws_bytes, int32_t* dev_status, void* stream);

/*
 * observe: statistics of one verify cycle for offline analysis ([SGLang]
 * "observability": the acceptance ceiling that cap-accept exposes, the
 * per-request confidences and calibration metrics such as ECE; [DSpark
 * notes] sec. 8.1: position d counts only where positions 1..d-1 were all
 * accepted).  Position d = 1..gamma of request i is observed when
 * d <= min(A_i + 1, w_i), A_i = ceiling[i], w_i = cu[i+1] - cu[i] - 1; its
 * outcome is hit = (d <= A_i).
 * In:  conf [R, gamma] fp32 (the confidences the scheduler ranked),
 *      cu_seqlens [R+1] of the verify, ceiling [R] (sdm_verify's ceiling: the
 *      acceptance count of the whole verified window), cls [R] class ids in
 *      [0, n_class), n_bins >= 1.
 * Out (device): hist [n_class, gamma+1] int32: requests per class and
 *      ceiling; reached, hits [n_class, gamma] int32: observed positions and
 *      their hits per class and position; bin_n, bin_hit [n_bins] int32 and
 *      bin_conf [n_bins] fp64: per equal-width bin the observations, hits and
 *      the sum of the confidences (c clamped to [0, 1], NaN as 0, in bin
 *      floor(c n_bins) of an fp32 product, c = 1 in the top bin); ece [1]
 *      fp64 = sum_b |bin_hit_b - bin_conf_b| / N, N = sum_b bin_n_b (0 when
 *      N = 0).  bin_conf is summed by atomic adds: its last bits may differ
 *      between runs; the counts are exact.
 * Limits: 4 n_class (3 gamma + 1) + 16 n_bins <= 49152 bytes, else
 *      SDM_ERR_UNSUPPORTED.
 * Device checks: a class id outside [0, n_class) sets SDM_DEV_BAD_CLASS and
 * the request is skipped; a window outside [0, gamma] or a ceiling outside
 * [0, w_i] sets SDM_DEV_BAD_WINDOW and is clamped.
 */
sdm_status sdm_observe(const float* conf, const int32_t* cu_seqlens, const int32_t* ceiling, const int32_t* cls, int R,
                       int gamma, int n_class, int n_bins, int32_t* hist, int32_t* reached, int32_t* hits,
                       int32_t* bin_n, int32_t* bin_hit, double* bin_conf, double* ece, int32_t* dev_status,
                       void* stream);

/*
 * Paged key/value cache of one attention layer: the state that the target
 * forward between pack and verify reads and extends ([SGLang] "ragged verify"
 * packs the rows; the cache itself is the serving engine's and has no
 * counterpart on the pages).
 *
 * Token t of request i lives in slot t % page of page table[i, t / page].
 * Pools are [n_pages, kv_heads, page, head_dim], K and V apart, in bf16 or
 * e4m3.  An e4m3 cache holds one scale per token and kv head, a power of two:
 * k_exp / v_exp [n_pages, kv_heads, page] hold its exponent + 127, and the
 * value that a code stands for is code * 2^(exp - 127) in bf16: exact for what
 * cache_write leaves (17 to 246), rounded for what else a caller may put there
 * (0 and 255 are read as 1 and 254).
 * Constraints: head_dim 64 or 128; page 16, 32, 64 or 128; n_pages * kv_heads
 * * page < 2^31; pools and exponents 16-byte aligned.  Else
 * SDM_ERR_UNSUPPORTED.
 *
 * The operations below take each request's committed length ctx_len[i] and
 * its window of new tokens: rows cu_seqlens[i] .. cu_seqlens[i+1] - 1 of the
 * packed arrays (sdm_pack_ragged's layout; a tree's window is its N + 1 slots)
 * sit at tokens ctx_len[i], ctx_len[i] + 1, ....  `rows` is the packed arrays'
 * row count, an upper bound on cu_seqlens[R]; rows that no window holds are
 * neither read nor written, and with rows = 0 the packed arrays may be NULL.  Device checks (OR-ed into *dev_status): a window
 * that is not within [0, rows] or not monotone counts as empty, a negative
 * ctx_len as 0 (SDM_DEV_BAD_WINDOW); tokens past max_pages * page, or past
 * 2^31 - 256, are left out, and a token whose page id is outside [0, n_pages)
 * is skipped when written and moved, read back as zeros, and as page 0 by
 * sdm_attend (SDM_DEV_BAD_PAGE).
 */
typedef struct {
    void* k;              /* device pool */
    void* v;
    uint8_t* k_exp;       /* e4m3 only, else NULL */
    uint8_t* v_exp;
    const int32_t* table; /* device [R, max_pages] page ids */
    int32_t dtype;        /* SDM_BF16 or SDM_E4M3 */
    int32_t n_pages;
    int32_t kv_heads;
    int32_t page;         /* tokens per page */
    int32_t head_dim;
    int32_t max_pages;    /* columns of table */
} sdm_cache;

/*
 * cache_write: the window's keys and values into their slots.  e4m3: per
 * token and kv head x[head_dim], e = the least integer in [-110, 119] with
 * max |x| <= 448 * 2^e over the finite elements; code = x * 2^-e rounded to
 * the nearest e4m3 value, ties to even, cut at +-448; a NaN or infinity is
 * stored as NaN.
 * In:  cache (host struct; its pools are written), k, v [rows, kv_heads,
 *      head_dim] bf16 with k_stride / v_stride elements from row to row (a
 *      multiple of 8, at least kv_heads * head_dim; bases 16-byte aligned: a
 *      slice of a fused projection's output will do), cu_seqlens [R+1],
 *      ctx_len [R].
 * Here and in cache_read R, rows <= 2^31 - 2^16.
 * Slots of different tokens must differ (they do when no two requests share
 * a page they write).
 */
sdm_status sdm_cache_write(const sdm_cache* cache, const uint16_t* k, const uint16_t* v, int64_t k_stride,
                           int64_t v_stride, const int32_t* cu_seqlens, const int32_t* ctx_len, int R, int rows,
                           int32_t* dev_status, void* stream);

/*
 * cache_read: tokens back as bf16 rows (exactly the values held).  Request
 * i's tokens first[i], first[i] + 1, ... fill rows cu_rows[i] .. cu_rows[i+1]
 * - 1 of k_out, v_out [rows, kv_heads, head_dim] (first NULL: from token 0).
 */
sdm_status sdm_cache_read(const sdm_cache* cache, const int32_t* cu_rows, const int32_t* first, int R, int rows,
                          uint16_t* k_out, uint16_t* v_out, int32_t* dev_status, void* stream);

/*
 * cache_commit: after sdm_verify_tree, the accepted path's keys, values and
 * scales move from their tree slots to follow the committed tokens, so that
 * the next window can start there.  path[i, 0] = 0 (the root) and path[i, j]
 * = the lowest slot c > path[i, j-1] whose parent is path[i, j-1] and whose
 * token is out_tok[i, j-1], j = 1..accept[i]; token ctx_len[i] + path[i, j]
 * moves to ctx_len[i] + j.  (A chain's accepted drafts are a prefix of its
 * window and need no move.)
 * In:  tok, parent [R, N+1], n_nodes [R] (sdm_draft_tree), out_tok [R, B+1],
 *      accept [R] (sdm_verify_tree), ctx_len [R].  N < 16384, B <= 16384.
 * Out: path [R, B+1] int32 (-1 past the path); length [R] = ctx_len +
 *      accepted + 1, the next ctx_len (may be NULL; may be ctx_len itself).
 * A path that breaks off (no such slot) is cut there: SDM_DEV_BAD_TOKEN.
 */
sdm_status sdm_cache_commit(const sdm_cache* cache, const int32_t* tok, const int32_t* parent,
                            const int32_t* n_nodes, const int32_t* out_tok, const int32_t* accept,
                            const int32_t* ctx_len, int R, int N, int B, int32_t* path, int32_t* length,
                            int32_t* dev_status, void* stream);

/*
 * attend: attention of every window row over its request's cached tokens,
 * the window's own among them (write them first).  For row p of request i,
 * query head h, kv head h / (H / kv_heads):
 *     s_j = scale * q . k_j over the tokens j that the row sees
 *     out = sum_j softmax(s)_j v_j,   lse = log sum_j exp(s_j)
 * The row's position is t = ctx_len[i] + p.  It sees the tokens j <= t with
 * t - j < window or j < sinks (window <= 0: all j <= t).  With tree_mask (the
 * mask of sdm_draft_tree, [R, tree_nodes, words], words = ceil(tree_nodes /
 * 32): bit c of node p set if c is p or an ancestor) the window's tokens are
 * seen as the row's bits say, whatever their distance, and t = ctx_len[i] +
 * depth, depth = max(0, bits set - 1).  A row that sees nothing, or only
 * scores of -inf, gives out 0, lse -inf; one that sees a score of +inf and no
 * NaN gives out NaN, lse +inf.  What a row does not see does not touch its
 * result, NaN and infinities included.
 * In:  cache; q [rows, H, head_dim] bf16, q_stride elements from row to row
 *      (a multiple of 8, at least H * head_dim, base 16-byte aligned); H a
 *      multiple of kv_heads, at most 128 times it; cu_seqlens [R+1], ctx_len
 *      [R]; max_window: the longest window (a longer one is cut:
 *      SDM_DEV_BAD_WINDOW; with tree_mask at most tree_nodes); 0 < scale
 *      <= 2e38; sinks >= 0; R <= 16384.
 * Out: out [rows, H, head_dim] bf16; lse [rows, H] fp32 (may be NULL).
 * Scores, statistics and sums are fp32; the weights exp(s - m) are rounded to
 * bf16 for the second product (the tensor cores' operand type).  An output is
 * within 2^-8 |out| + 2^-8 sum_j softmax(s)_j |v_j| of the formula's, and the
 * fp32 sums' own error: the result's rounding and the weights'.  The second
 * part goes, because what the weights' rounding leaves is multiplied too,
 * where a request's rows of a kv head (query heads times window) see at most
 * 1152 keys, or 2048 if the rows are at most 64.
 * ws:  sdm_workspace_size(SDM_OP_ATTEND, R, max_window, H, head_dim, rows,
 *      kv_heads, 0).
 */
sdm_status sdm_attend(const sdm_cache* cache, const uint16_t* q, int64_t q_stride, const int32_t* cu_seqlens,
                      const int32_t* ctx_len, int R, int rows, int max_window, int H, float scale, int window,
                      int sinks, const int32_t* tree_mask, int tree_nodes, uint16_t* out, float* lse, void* ws,
                      size_t ws_bytes, int32_t* dev_status, void* stream);

/*
 * qk_rotate: what stands between the projections and the cache: every query
 * and key head vector x normalised, y = x / sqrt(mean(x^2) + eps) * weight (no
 * weight: y = x), and rotated by its position: pair j < rot_dim / 2 by the
 * angle position * freq[j], (a, b) -> (a cos - b sin, b cos + a sin).  A pair is
 * elements (j, j + rot_dim / 2), or (2 j, 2 j + 1) if interleaved; elements
 * from rot_dim on are not rotated.  With a cache the keys, and the values as
 * they are, go into its slots as by sdm_cache_write (the same bits as rotating
 * into k_out and writing that); without one the keys go to k_out.
 * The row at window position p of request i has the position start[i] + p, or
 * start[i] + row_pos[row] (a tree's depths; sdm_pack_ragged's packed_pos);
 * start NULL: ctx_len[i].  start differs from ctx_len where tokens were
 * evicted.  Positions are exact to 2^53; the angle is reduced in fp64.
 * In:  q [rows, H, head_dim], k [rows, kv_heads, head_dim], v (with a cache)
 *      the same, bf16, strides in elements from row to row (multiples of 8,
 *      at least a row, bases 16-byte aligned); q_weight, k_weight [head_dim]
 *      fp32, 16-byte aligned, or NULL; eps >= 0; freq [rot_dim / 2] fp64
 *      radians per token (NULL with rot_dim 0); rot_dim a multiple of 8, at
 *      most head_dim; head_dim 64 or 128, and the cache's; kv_heads likewise;
 *      cu_seqlens, ctx_len as in sdm_cache_write (without a cache ctx_len may
 *      be NULL if start is given); R <= 2^31 - 2^16, rows * (H + 2 kv_heads)
 *      < 2^31.
 * Out: q_out, and k_out without a cache (NULL with one): rows with strides of
 *      their own; each may be its input.  Rows that no window holds are left
 *      as they were; one that several hold (offsets that are not monotone) is
 *      rotated for one of them.  fp32 throughout, rounded to bf16 once (so a
 *      vector whose sum of squares passes fp32, with elements beyond 10^18,
 *      is normalised to zeros).
 * Device checks as in sdm_cache_write; a row whose page is bad still has its
 * query rotated, one past the page table is left out.
 */
sdm_status sdm_qk_rotate(const sdm_cache* cache, const uint16_t* q, int64_t q_stride, int H, const uint16_t* k,
                         int64_t k_stride, const uint16_t* v, int64_t v_stride, int kv_heads, int head_dim,
                         const float* q_weight, const float* k_weight, float eps, const double* freq, int rot_dim,
                         int interleaved, const int32_t* cu_seqlens, const int32_t* ctx_len, const int32_t* start,
                         const int32_t* row_pos, int R, int rows, uint16_t* q_out, int64_t q_out_stride,
                         uint16_t* k_out, int64_t k_out_stride, int32_t* dev_status, void* stream);

/*
 * token_logprobs: what a served request wants to know of its tokens, after
 * sdm_verify or sdm_verify_tree.  Position p < n[i] of request i, with its
 * target row z (row cu_seqlens[i] + p, or cu_seqlens[i] + path[i, p]) and
 * token y = tok[i, p], has
 *     logp = log softmax(z / T)[y],     entropy = -sum_v P_v log P_v,
 *     rank = tokens ahead of y: a greater logit, or an equal one and a lower id,
 *     top_tok, top_logp = the `top` first tokens in that order, and theirs.
 * A tree's target [R, N+1, V] has cu_seqlens[i] = i (N + 1) and the path that
 * sdm_cache_commit returns; a prompt is one window whose tok are its next tokens.
 * In:  target [row_capacity, V] (dtT), cu_seqlens [R+1], path [R, W] or NULL,
 *      tok [R, W] (sdm_verify's out_tok), n [R] (its n_out) or NULL: every row
 *      of the windows, W at most.  V % 8 == 0, V >= 8, target 16-byte aligned;
 *      R W <= 2^27; 0 <= top <= min(32, V); log2(e) / T within 1e-8 .. 1e8.
 * Out: logp [R, W] fp32; entropy fp32, rank int32 [R, W] (each may be NULL);
 *      top_tok int32, top_logp fp32 [R, W, top] (NULL if top = 0).  Positions
 *      from n[i] on are left as they were.
 * Sums are fp32 relative to a reference near the maximum.  A logit of -inf has
 * logp -inf; a row of nothing else, or with a NaN, has logp and entropy NaN (a
 * NaN has some rank, and is listed as if it were -inf), one with +inf logp
 * -inf but for those NaN, entropy NaN.
 * Device checks: n[i] outside [0, W] (cut), a row outside its window
 * (SDM_DEV_BAD_WINDOW) or past row_capacity (SDM_DEV_CAPACITY): left out; a
 * token outside [0, V) has logp -inf and rank V (SDM_DEV_BAD_TOKEN).
 */
sdm_status sdm_token_logprobs(const void* target, sdm_dtype dtT, int row_capacity, int V, const int32_t* cu_seqlens,
                              const int32_t* path, const int32_t* tok, const int32_t* n, int R, int W,
                              float temperature, int top, float* logp, float* entropy, int32_t* rank,
                              int32_t* top_tok, float* top_logp, int32_t* dev_status, void* stream);

/*
 * attend_weight: the attention weight that each cached token got from the
 * committed rows of a call, per kv head, for sdm_cache_evict.  After
 * sdm_attend (its lse) and, for trees, sdm_cache_commit (the keys have to be
 * where they stay):
 *     mass_out[i, g, j] = (j < ctx_len[i] ? mass[i, g, j] : 0)
 *                         + sum_{p, h} exp(scale q . k_j - lse)
 * over the rows p < count[i] that see token j and the query heads h of kv head
 * g, for j < ctx_len[i] + count[i]; later entries are left as they were.  Row
 * p is packed row cu_seqlens[i] + p, or cu_seqlens[i] + path[i, p] (count: the
 * path's length, root included), and sits at token ctx_len[i] + p; it sees j
 * <= ctx_len[i] + p within `window` or below `sinks`, as in sdm_attend.
 * In:  cache (its values are not read); q and q_stride as in sdm_attend; lse
 *      [rows, H] fp32; cu_seqlens [R+1], ctx_len [R]; count [R] or NULL (whole
 *      windows); path [R, path_stride] or NULL, path_stride >= max_count;
 *      max_count: the largest count (larger ones are cut); mass [R, kv_heads,
 *      stride] fp32 or NULL (zeros), stride < 2^31; R <= 16384, H at most 128
 *      kv_heads.
 * Out: mass_out, the same shape; may be mass.
 * Scores and sums are fp32, in an order that depends on the sizes alone.  A
 * row whose lse is -inf or NaN adds nothing; a score of +inf or NaN beside an
 * lse of +inf, and infinities in q over an e4m3 cache, count as NaN.
 * ws:  sdm_workspace_size(SDM_OP_ATTEND_WEIGHT, R, max_count, H, head_dim, rows,
 *      kv_heads, 0) bytes.
 * Device checks as in sdm_attend; a count outside [0, max_count] or past the
 * window is cut, a row of the path outside the window adds nothing
 * (SDM_DEV_BAD_WINDOW); tokens past `stride` are left out (SDM_DEV_BAD_PAGE).
 */
sdm_status sdm_attend_weight(const sdm_cache* cache, const uint16_t* q, int64_t q_stride, const float* lse,
                             const int32_t* cu_seqlens, const int32_t* ctx_len, const int32_t* count,
                             const int32_t* path, int path_stride, int R, int rows, int max_count, int H, float scale,
                             int window, int sinks, const float* mass, float* mass_out, int64_t stride, void* ws,
                             size_t ws_bytes, int32_t* dev_status, void* stream);

/*
 * cache_evict: every request's cache cut to `keep` tokens, chosen for each kv
 * head by itself: the positions below `sinks` and the last `recent` ones
 * first, then those of the largest weight (equals: the lowest slot; a NaN
 * last).  Request i holds n = ctx_len[i] + count[i] tokens; slot s < ctx_len[i]
 * has the position pos[i, g, s] that an earlier cut left, slot ctx_len[i] + j
 * the position start[i] + j.  A kept token in front of slot `keep` stays in its
 * slot; the j-th of the others, in order, moves (key, value, scales, weight and
 * position) to the j-th slot that becomes free there.  A request with n <= keep
 * keeps all.  Keys carry their rotation, so a cache in another order attends
 * alike; sdm_attend's `window` and `sinks` go by slots, so use neither then.
 * In:  cache (its pools are written, in any page that holds one of a request's
 *      n tokens: no other request may use that page, so a common prompt's are
 *      copied first); mass, pos [R, kv_heads, stride] (pos is not read from
 *      ctx_len on), stride < 2^31 (the blocks' number and shared memory follow
 *      it: 64 full caches of 2048 and 8 heads take 13 us with a stride of 2300,
 *      30 with 30000, 150 with 100000);
 *      ctx_len [R]; count [R] or NULL (0); start [R] or NULL (ctx_len: nothing
 *      was evicted yet); 0 <= sinks, recent, sinks + recent <= keep, keep >= 1;
 *      R * kv_heads <= 2^24.
 * Out: mass_out, pos_out [R, kv_heads, stride], filled below length[i], entries
 *      from there on left as they were; may be mass and pos.  length [R] =
 *      min(n, keep), the next ctx_len; next [R] (may be NULL) = start + count,
 *      the next start.  Neither may be an input: a request's heads read those
 *      beside one another.
 * ws:  sdm_workspace_size(SDM_OP_CACHE_EVICT, R, kv_heads, 0, 0, stride, 0, keep).
 * Device checks: a negative ctx_len or count as 0 (SDM_DEV_BAD_WINDOW); tokens
 * past the page table or `stride` are left out, a row whose page is bad is not
 * moved (SDM_DEV_BAD_PAGE).
 */
sdm_status sdm_cache_evict(const sdm_cache* cache, const float* mass, const int32_t* pos, int64_t stride,
                           const int32_t* ctx_len, const int32_t* count, const int32_t* start, int R, int keep,
                           int sinks, int recent, float* mass_out, int32_t* pos_out, int32_t* length, int32_t* next,
                           void* ws, size_t ws_bytes, int32_t* dev_status, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* SDM_H */
