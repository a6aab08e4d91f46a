/*
 * qcf.h -- C ABI of a GB300 (sm_103a) library for query-centric KV-cache fusion
 * in retrieval-augmented prefill.
 *
 * The method (QCFuse: Query-Centric Cache Fusion for Efficient RAG Inference,
 * technical summary, section 2 "Methodology"; CacheBlend's selective recompute
 * as described in "KVCache reuse 01", section 1.3):
 *   offline  each retrieved chunk is prefilled alone at positions 0..L-1 and its
 *            per-layer K/V kept in host memory; a few tokens of largest key norm
 *            per chunk are kept as anchors;
 *   online   the query runs the first layers with the anchors as a KV prefix,
 *            one critical middle layer's keys are scored by the query's softmax
 *            attention mass, the top-N context tokens are selected, and layer by
 *            layer only those rows (plus the query) are recomputed, attending to
 *            the fused cache with causality by true position, while the next
 *            layer's chunk K/V streams in from host memory.
 *
 * Conventions (every entry point):
 *  - Returns qcf_status.  Argument errors are reported synchronously before any
 *    launch; the message of the last error on the calling thread is returned by
 *    qcf_last_error().  No C++ exception crosses this boundary.
 *  - Pointers are device memory owned by the caller unless documented as host
 *    (pageable or pinned).  The library never allocates device memory on these
 *    paths and never frees caller memory.  Scratch comes from the caller as
 *    (ws, ws_bytes), sized by the matching *_workspace_size() function, 256-byte
 *    aligned; too small gives QCF_ERR_WORKSPACE.
 *  - Work is enqueued asynchronously on the caller's CUDA stream, passed as
 *    void* (a cudaStream_t; NULL is the legacy default stream).
 *  - Device-side failures (a bounded wait that ran out, an index that failed a
 *    check) set bits of a device status word instead of trapping; read and clear
 *    it with qcf_query_status() after synchronising.
 *  - Tensors are row-major and contiguous: K/V caches are [rows][H_kv][D], query
 *    blocks [rows][H_q][D], hidden states [rows][d].  bf16 buffers are passed as
 *    qcf_bf16 (the raw 16-bit pattern).  Base pointers must be 16-byte aligned
 *    (QCF_ERR_ALIGN otherwise).
 *  - Supported head dims D: 16, 64, 128.  H_q must be a multiple of H_kv.
 *  - Indices and positions are int32; position tables are strictly ascending.
 */
#ifndef QCF_H_
#define QCF_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef uint16_t qcf_bf16;

typedef enum qcf_status {
  QCF_OK = 0,
  QCF_ERR_INVALID_ARG = 1,  /* null pointer, negative size, bad enum */
  QCF_ERR_SHAPE = 2,        /* sizes inconsistent or outside the supported set */
  QCF_ERR_ALIGN = 3,        /* pointer or stride not 16-byte aligned */
  QCF_ERR_WORKSPACE = 4,    /* ws_bytes smaller than the *_workspace_size() */
  QCF_ERR_CUDA = 5,         /* a CUDA runtime/driver call failed */
  QCF_ERR_TIMEOUT = 6,      /* a device-side bounded wait ran out */
  QCF_ERR_UNSUPPORTED = 7,  /* no sm_103a device, or a feature not built */
  QCF_ERR_DEVICE = 8        /* a device-side index check failed */
} qcf_status;

/* Device status word bits (qcf_query_status). */
#define QCF_DEV_TIMEOUT 0x1u
#define QCF_DEV_BAD_INDEX 0x2u
#define QCF_DEV_NO_PAGES 0x4u

/* ------------------------------------------------------------------ library */

/* Message of the last error on this thread ("" when none). Never NULL. */
const char* qcf_last_error(void);
/* Version string of the library build. */
const char* qcf_version(void);
/* Reads and clears the device status word (bits QCF_DEV_*), synchronising
 * `stream` first.  *status = 0 means no device-side failure was seen. */
qcf_status qcf_query_status(void* stream, uint32_t* status);
/* Host-side fault injection for tests: the next call of the given kind fails
 * before launching anything.  0 clears.  Kinds: 1 = invalid index table,
 * 2 = short workspace, 3 = failed host-to-device copy, 4 = misaligned pointer. */
qcf_status qcf_debug_set_fault(int kind);
/* Enables device-side index checks (positions ascending and in range) in the
 * kernels that read index tables; failures set QCF_DEV_BAD_INDEX. */
qcf_status qcf_set_check(int on);
/* Total kernel launches issued by the library since load (all entry points). */
int64_t qcf_launch_count(void);

/* Per-kernel timing with CUDA events recorded around each launch on the
 * launching stream.  Enable, run, then read: names/ms/launches of up to `max`
 * kernel classes; reading synchronises on the recorded events and resets. */
qcf_status qcf_timing_enable(int on);
qcf_status qcf_timing_read(int max, const char** names, double* ms, int64_t* launches, int* n_classes);

/* Measures the special-function unit's exp2 throughput of the current device (exp2 per
 * second over all SMs): eight independent chains of ex2.approx per thread, the best of
 * two timed launches after one warm-up.  The ceiling of the critical-layer profile, which
 * evaluates two exponentials per score-row element.  scratch: device memory of at least
 * num_SMs * 8 * 256 * 4 bytes (the kernel's outputs).  Synchronises the stream. */
qcf_status qcf_calibrate_exp2_rate(float* scratch, size_t scratch_bytes, double* per_second, void* stream);

/* ------------------------------------------------------------------ shapes */

/* N = ceil(ratio * C) for a recompute ratio in basis points (1500 = 15 %),
 * computed in integers and clamped to [0, C]: the number of context tokens
 * recomputed (Cache-Craft's N = ceil(CFO * |C_i|), "KVCache reuse 01" 2.3.3). */
qcf_status qcf_num_selected(int C, int ratio_bp, int* N);

/* RoPE tables, rotate-half convention: pair (k, k + D/2) of a head at position p
 * turns by angle p * theta^(-2k/D).  cos/sin are device [max_pos][D/2] fp32. */
typedef struct qcf_rope_table {
  const float* cos;
  const float* sin;
  int max_pos;
  int head_dim;
} qcf_rope_table;

/* Fills host buffers cos_host/sin_host [max_pos][D/2] with the angles taken in
 * fp64 and rounded to fp32 (the caller copies them to the device). */
qcf_status qcf_rope_table_fill_host(float* cos_host, float* sin_host, int max_pos, int D, double theta);

/* ------------------------------------------------------------------ offline */

/* Semantic-summary anchors (QCFuse 2.A "Anchor-based Lightweight Query
 * Probing"): for each chunk, the n_anchor tokens whose key has the largest L2
 * norm over all H_kv*D entries, ties to the lower index, written ascending and
 * chunk-local to anchor_idx [n_chunks][n_anchor].
 *   K            device [C][Hkv][D] bf16, the critical layer's stored keys
 *   chunk_start  HOST [n_chunks + 1], ascending, chunk_start[n_chunks] = C;
 *                every chunk needs length >= n_anchor and <= 16384
 *   norms        device [C] fp32 key norms, or NULL
 * Norms are accumulated in fp32. */
qcf_status qcf_anchor_keynorm_topk(const qcf_bf16* K, const int32_t* chunk_start, int n_chunks,
                                   int Hkv, int D, int n_anchor, int32_t* anchor_idx, float* norms,
                                   void* stream);

/* ------------------------------------------------------------------ online steps */

/* Re-rotation of reused keys to their new absolute positions ("adjust the
 * positional encoding" of chunks not at the prefix, CacheBlend problem
 * definition 2.4): row i of segment s becomes R(delta[s]) * K_src[i].
 *   K_src, K_dst  device [n_rows][Hkv][D] bf16; may be the same buffer (in place)
 *   seg_start     HOST [n_seg + 1] ascending, seg_start[n_seg] = n_rows
 *   seg_delta     HOST [n_seg], 0 <= delta < t->max_pos
 * Rotation in fp32 from the fp32 table, rounded to bf16. */
qcf_status qcf_rope_reposition(const qcf_bf16* K_src, qcf_bf16* K_dst, int64_t n_rows, int Hkv, int D,
                               const int32_t* seg_start, const int32_t* seg_delta, int n_seg,
                               const qcf_rope_table* t, void* stream);

/* Critical-layer attention profiling (QCFuse 2.A "Critical-layer Attention
 * Profiling"): score[j] = sum over query rows r and heads h of
 * softmax_j(scale * q[r,h] . K[j, h / (Hq/Hkv)]) over the C context keys.
 *   q       device [nq][Hq][D] bf16
 *   K       device [C][Hkv][D] bf16 (already re-rotated)
 *   scores  device [C] fp32
 * Products on tensor cores (fp32 accumulate), softmax in fp32 with exact
 * per-row max and normaliser (two passes over K). */
size_t qcf_profile_scores_workspace_size(int nq, int C, int Hq, int Hkv, int D);
qcf_status qcf_profile_scores(const qcf_bf16* q, const qcf_bf16* K, int nq, int C, int Hq, int Hkv, int D,
                              float scale, float* scores, void* ws, size_t ws_bytes, void* stream);

/* qcf_profile_scores with no caller workspace and no allocation of any kind.
 * The pages have no counterpart: this exists for callers that cannot allocate
 * device memory at the point of the call -- for example a serving loop that
 * gave all free device memory to its KV-cache pool at start-up, or code holding
 * a memory budget fixed in advance that must not call cudaMalloc (which may
 * also synchronise the device) on the request path.
 * Scratch is one fixed 8 MiB array in device global memory, present on every
 * GPU that loads the library for the life of the process.  A shape whose
 * qcf_profile_scores_workspace_size() exceeds 8 MiB is rejected with
 * QCF_ERR_WORKSPACE before anything runs; the 8B-shaped request (64 query rows
 * x 32 heads over 5120 keys) needs under 1 MiB and 131072 keys under 6 MiB.
 * The first call on each device looks up the array's device address (with that
 * device current); make that first call before any stream capture.  All calls
 * share the one array: calls that overlap on the GPU (different streams, or
 * host threads without ordering) race and corrupt each other's results.  Every
 * call rewrites all the scratch it reads, so no clearing is needed.
 * Arguments, layouts and results are those of qcf_profile_scores. */
qcf_status qcf_profile_scores_noalloc(const qcf_bf16* q, const qcf_bf16* K, int nq, int C, int Hq, int Hkv, int D,
                                      float scale, float* scores, void* stream);

/* Top-N selection (QCFuse 2.A: "the Top-N context token indices"): the indices of
 * the N largest scores, ties to the lower index (the order of a stable sort by
 * descending score), written ascending to sel [N].  0 <= N <= C <= 2^24.
 * Exact on the fp32 bit patterns; -0.0 counts as +0.0; scores must not be NaN. */
qcf_status qcf_topn_select(const float* scores, int C, int N, int32_t* sel, void* stream);

/* Top-N selection with scratch, for long score vectors: the same result as
 * qcf_topn_select.  Above 16384 scores the work spreads over a cooperative grid of
 * up to one CTA per SM (4096 scores each) that reads the scores once and meets at
 * bounded grid barriers (a barrier that runs out sets QCF_DEV_TIMEOUT and leaves sel
 * incomplete); at or below 16384 scores, or beyond what one resident grid covers,
 * this is qcf_topn_select and ws is not touched.
 *   ws  device scratch of qcf_topn_select_workspace_size(C) bytes (0 for C <= 16384,
 *       then ws may be NULL); it needs no clearing (each call resets the state it
 *       uses, on the GPU); calls that overlap on the GPU need separate scratch. */
size_t qcf_topn_select_workspace_size(int C);
qcf_status qcf_topn_select_ws(const float* scores, int C, int N, int32_t* sel, void* ws, size_t ws_bytes,
                              void* stream);

/* KV deviation of recomputed rows ("KVCache reuse 01" 1.3.2, "KV Deviation"): for i < n,
 * dev[i] = sum over the Hkv*D entries of (k_new[i] - K_cache[pos[i]])^2 + (v_new[i] - V_cache[pos[i]])^2,
 * fp32 accumulation of bf16 inputs.
 *   k_new, v_new  device [n][Hkv][D] bf16 (fresh rows); pos device [n] in [0, T)
 *   K_cache, V_cache device [T][Hkv][D] bf16 (the reused rows); dev device [n] fp32.
 * A position outside [0, T) gives dev 0 and sets QCF_DEV_BAD_INDEX in the device status word. */
qcf_status qcf_kv_deviation(const qcf_bf16* k_new, const qcf_bf16* v_new, const int32_t* pos, int n,
                            const qcf_bf16* K_cache, const qcf_bf16* V_cache, int T, int Hkv, int D, float* dev,
                            void* stream);

/* Gathers the rows of the tokens chosen for recompute ("KVCache reuse 01" 1.3.4,
 * selective recompute flow: the selected tokens are masked out of the full
 * input and only they run through the layer): dst[i][:] = src[idx[i]][:] for i < n.
 *   src  device [src_rows][width] bf16 (width % 8 == 0); dst device [n][width] bf16
 *   idx  device [n], each in [0, src_rows); an index outside that range is not read:
 *        its dst row is left as it was and QCF_DEV_BAD_INDEX is set in the status word. */
qcf_status qcf_gather_rows(const qcf_bf16* src, int64_t src_rows, int width, const int32_t* idx, int n,
                           qcf_bf16* dst, void* stream);

/* Writes fresh K/V rows of the recomputed tokens into the fused cache at their
 * positions ("KVCache reuse 01" 1.3.4: the recomputed K_i, V_i extend the reused
 * cache, and attention then runs over all tokens of the layer):
 * K_cache[pos[i]] = k_new[i], V_cache[pos[i]] = v_new[i].
 *   k_new, v_new  device [n][Hkv][D] bf16; pos device [n] in [0, T), distinct. */
qcf_status qcf_scatter_kv(const qcf_bf16* k_new, const qcf_bf16* v_new, const int32_t* pos, int n, int Hkv,
                          int D, qcf_bf16* K_cache, qcf_bf16* V_cache, int T, void* stream);

/* Location-aware sparse causal attention (QCFuse 2.A: a discrete token index
 * table, causal constraint by true position): for each recomputed row i at
 * position pos[i], o[i,h] = sum_{j <= pos[i]} softmax_j(scale * q[i,h] . K[j,g]) V[j,g]
 * with g = h / (Hq/Hkv), over the fused cache (reused rows plus fresh rows).
 *   q    device [n][Hq][D] bf16;  pos device [n] strictly ascending, < T
 *   K,V  device [T][Hkv][D] bf16; o device [n][Hq][D] bf16
 *   lse  device [n][Hq] fp32 natural-log sum of exp of the scaled logits, or NULL
 * Tensor-core QK^T and PV (fp32 accumulate), online softmax in fp32. */
size_t qcf_sparse_causal_attn_workspace_size(int n, int T, int Hq, int Hkv, int D);
qcf_status qcf_sparse_causal_attn(const qcf_bf16* q, const int32_t* pos, int n, const qcf_bf16* K,
                                  const qcf_bf16* V, int T, int Hq, int Hkv, int D, float scale, qcf_bf16* o,
                                  float* lse, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------ dense pieces */

/* out = A * W^T for A device [M][K] bf16 and W device [N][K] bf16 (nn.Linear
 * layout) on tcgen05 tensor cores with TMEM accumulators.
 *   epilogue QCF_EPI_STORE_BF16: out is bf16 [M][N]
 *   epilogue QCF_EPI_ADD_F32:    out is fp32 [M][N] and receives out += A W^T
 *   | QCF_LINEAR_W_KN:           W is stored [K][N] instead (out = A * W)
 * K % 64 == 0, N % 64 == 0.  ws: device scratch of qcf_linear_workspace_size
 * bytes (tile counters and fp32 partial sums when the planner shares output
 * tiles between CTAs); its contents need not survive between calls, but calls
 * that share it must be ordered on one stream.  Results are bitwise repeatable
 * for the same inputs and shapes (partial sums are added in a fixed order). */
#define QCF_EPI_STORE_BF16 0
#define QCF_EPI_ADD_F32 1
#define QCF_LINEAR_W_KN 0x10
size_t qcf_linear_workspace_size(int M, int N, int K);
qcf_status qcf_linear(const qcf_bf16* A, int M, int K, const qcf_bf16* W, int N, int epilogue, void* out,
                      void* ws, size_t ws_bytes, void* stream);

/* h = x / sqrt(mean(x^2) + eps) * g per row; x device fp32 [n][d], g bf16 [d],
 * h bf16 [n][d].  Statistics in fp32. */
qcf_status qcf_rmsnorm(const float* x, int n, int d, const qcf_bf16* g, float eps, qcf_bf16* h, void* stream);

/* ------------------------------------------------------------------ model */

typedef struct qcf_dims {
  int n_layers, d_model, n_heads, n_kv_heads, head_dim;
  int ffn;         /* FFN width of the model */
  int ffn_padded;  /* ffn rounded up to a multiple of 64 (zero rows/columns) */
  int vocab;
  float eps;
  float theta;
} qcf_dims;

/* One decoder layer's weights, device bf16, packed for the tensor-core GEMMs:
 *   w_qkv   [(Hq + 2 Hkv) D][d]   rows W_q, then W_k, then W_v
 *   w_o     [d][Hq D]
 *   w_gu    [2 ffn_padded][d]     blocks of 64 gate rows then the same 64 up rows
 *   w_down  [d][ffn_padded]       columns beyond ffn are zero
 *   g_attn, g_mlp [d]             RMSNorm gains */
typedef struct qcf_layer_weights {
  const qcf_bf16* w_qkv;
  const qcf_bf16* w_o;
  const qcf_bf16* w_gu;
  const qcf_bf16* w_down;
  const qcf_bf16* g_attn;
  const qcf_bf16* g_mlp;
} qcf_layer_weights;

typedef struct qcf_model {
  qcf_dims dims;
  const qcf_bf16* embed;            /* device [vocab][d] */
  const qcf_bf16* lm_head;          /* device [vocab][d] */
  const qcf_bf16* g_final;          /* device [d] */
  const qcf_layer_weights* layers;  /* HOST array [n_layers] */
  qcf_rope_table rope;              /* max_pos must exceed every position used */
} qcf_model;

/* One decoder layer for n recomputed rows (the selective recompute flow of
 * "KVCache reuse 01" 1.3.4): RMSNorm -> QKV GEMM with RoPE at rope_pos and the
 * fresh K/V written into the cache at cache_row (before attention) -> sparse
 * causal attention of row i over cache rows <= cache_row[i] -> O GEMM added to
 * x -> RMSNorm -> gate/up GEMM with SwiGLU -> down GEMM added to x.
 *   x          device fp32 [n][d], the residual stream, updated in place
 *   rope_pos   device [n] absolute positions (RoPE phase)
 *   cache_row  device [n] strictly ascending rows of the cache written and used
 *              as each row's causal bound (equal to rope_pos on the fused path)
 *   K_cache, V_cache device [T][Hkv][D] bf16 */
size_t qcf_layer_workspace_size(const qcf_dims* dims, int n, int T);
qcf_status qcf_fused_layer_forward(const qcf_model* m, int layer, float* x, const int32_t* rope_pos,
                                   const int32_t* cache_row, int n, qcf_bf16* K_cache, qcf_bf16* V_cache,
                                   int T, void* ws, size_t ws_bytes, void* stream);

/* Full recompute of T tokens at positions 0..T-1 ("Full KV Recompute",
 * CacheBlend problem definition 2.2): per-layer K/V into K_layers[l]/V_layers[l]
 * (HOST arrays of n_layers device pointers, each [T][Hkv][D]), the last row's
 * logits (device fp32 [vocab]) and the first token (device int32, argmax with
 * the lowest index on ties).  ids device [T]. */
size_t qcf_full_prefill_workspace_size(const qcf_dims* dims, int T);
qcf_status qcf_full_prefill(const qcf_model* m, const int32_t* ids, int T, qcf_bf16* const* K_layers,
                            qcf_bf16* const* V_layers, float* last_logits, int32_t* first_token, void* ws,
                            size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------ request driver */

/* A request: retrieved chunks in retrieval order, then the query.
 *   chunk_len       HOST [n_chunks]
 *   chunk_K/V_host  HOST arrays [n_chunks] of PINNED host pointers, each
 *                   [n_layers][chunk_len][Hkv][D] bf16 (post-RoPE at local positions)
 *   anchor_idx      HOST [n_chunks][n_anchor] chunk-local ascending
 *   anchor_K/V_host HOST arrays [n_chunks] of PINNED host pointers, each
 *                   [n_layers][n_anchor][Hkv][D] bf16 (the anchors' stored rows)
 *   ids             device [C + query_len]: chunk tokens in order, then the query
 *   forced_sel      device [N] ascending, or NULL to select by profiling */
typedef struct qcf_request {
  int n_chunks;
  const int32_t* chunk_len;
  const qcf_bf16* const* chunk_K_host;
  const qcf_bf16* const* chunk_V_host;
  int n_anchor;
  const int32_t* anchor_idx;
  const qcf_bf16* const* anchor_K_host;
  const qcf_bf16* const* anchor_V_host;
  const int32_t* ids;
  int query_len;
  int crit_layer;
  int ratio_bp;
  const int32_t* forced_sel;
  /* Appended fields: a zero-initialised request keeps the critical-layer selector. */
  int selector;                  /* QCF_SELECT_*; see below */
  const int32_t* layer_ratio_bp; /* HOST [L], QCF_SELECT_HKVD only: share of C kept after layer l, basis points,
                                    non-increasing, layer_ratio_bp[L-1] == ratio_bp */
} qcf_request;

/* Selectors (qcf_request.selector):
 *   QCF_SELECT_CRITICAL    QCFuse: probe layers 0..crit-1 with the anchor prefix, profile at crit_layer
 *                          (QCFuse 2.A); crit_layer = L-1 is the QCLast variant (QCFuse 4, "Results").
 *   QCF_SELECT_ALL_LAYERS  QCAll (QCFuse 4): the probe runs layers 0..L-2 (anchor stores must hold those
 *                          layers); the profile scores of every layer's query against that layer's
 *                          re-rotated keys are summed, then one top-N selection.  Every layer's keys must
 *                          land before the recompute starts: the cost the pages attribute to all-layer
 *                          profiling.  crit_layer still names the anchors' layer (chosen offline).
 *   QCF_SELECT_HKVD        CacheBlend's KV-deviation selection with gradual filtering ("KVCache reuse 01"
 *                          1.3.2-1.3.4): layer 0 projects K/V for every context token, layer l for the
 *                          tokens kept after layer l-1; a token's deviation is the squared L2 distance of
 *                          its fresh K and V to the reused (re-rotated) cache rows; the top
 *                          ceil(layer_ratio_bp[l] * C / 10000) by deviation (ties to the lower position)
 *                          are kept and get fresh K/V, attention and MLP at layer l with the query rows.
 *                          Anchors, crit_layer and forced_sel are ignored; out->scores gets layer 0's
 *                          deviation of every context token, out->sel the rows kept after the last layer. */
#define QCF_SELECT_CRITICAL 0
#define QCF_SELECT_ALL_LAYERS 1
#define QCF_SELECT_HKVD 2

/* Outputs: the fused cache of every layer (HOST arrays of device pointers
 * [C + Q][Hkv][D]), sel [N], scores [C], q_crit [Q][Hq][D] (nullable), the last
 * query row's logits [vocab], the first token on the device and, when
 * first_token_host (PINNED) is set, copied to the host on compute_stream. */
typedef struct qcf_outputs {
  qcf_bf16* const* K_layers;
  qcf_bf16* const* V_layers;
  int32_t* sel;
  float* scores;
  qcf_bf16* q_crit;
  float* last_logits;
  int32_t* first_token;
  int32_t* first_token_host;
  float* x_rows;  /* device fp32 [N + Q][d] final hidden states of the recomputed rows, or NULL */
  /* Appended: QCF_SELECT_HKVD only, or NULL.  device [L][N_0]: row l holds the N_l context rows kept
   * after layer l (ascending), N_l = ceil(layer_ratio_bp[l] * C / 10000). */
  int32_t* layer_sel;
} qcf_outputs;

/* The per-request fused prefill with the per-layer pipeline (QCFuse 2.A
 * "pipelined cache reconstruction"; the load/recompute pipeline of "KVCache
 * reuse 01" 1.3.5): anchors and the critical layer's keys are copied first, the
 * probe, profiling and top-N run, then layer l is recomputed on compute_stream
 * while later layers' chunk K/V are copied on copy_stream.  Enqueues only. */
size_t qcf_request_workspace_size(const qcf_dims* dims, int C, int Q, int n_anchor_total, int N);
/* Workspace for this particular request, any selector (QCF_SELECT_HKVD needs full-row buffers for
 * layer 0, which the size above does not cover).  0 when the request is malformed. */
size_t qcf_request_workspace_size_for(const qcf_dims* dims, const qcf_request* r);
qcf_status qcf_request_prefill(const qcf_model* m, const qcf_request* r, const qcf_outputs* out, void* ws,
                               size_t ws_bytes, void* compute_stream, void* copy_stream);

/* Storage tier (QCFuse 2.A: chunk KV kept on SSD, layer i+1 loaded while layer i is
 * recomputed; anchors stay in CPU memory).  qcf_request_prefill with the chunks' K/V read
 * from files instead of pinned host arrays (r->chunk_K_host / chunk_V_host are ignored;
 * the anchor stores are still host memory).  Per layer, a host function on the copy stream
 * reads that layer's keys and values of every chunk into one half of `staging` (pinned
 * host memory of qcf_storage_staging_bytes, page-aligned for files opened with O_DIRECT),
 * and the copy stream then copies them into the fused cache and re-rotates the keys; the
 * critical layer's keys are read first.  The read of layer l+2 reuses the half of layer l
 * after its copies completed, so reading overlaps the recompute of the layers already
 * landed, as in qcf_request_prefill.
 *   files[c]  chunk c's file: fd open for reading (not closed by the library); the keys of
 *             layer l, [len][Hkv][D] bf16, at k_offset + l * layer_stride, the values at
 *             v_offset + l * layer_stride.  With O_DIRECT, offsets and block sizes must
 *             meet the file system's alignment.
 * A failed or short read leaves that layer's rows undefined (no device fault) and is
 * reported, once the copy stream has run past it, by qcf_storage_status (the first
 * failure's errno since the last call, then cleared; 0 when none). */
typedef struct qcf_chunk_file {
  int fd;
  int64_t k_offset;
  int64_t v_offset;
  int64_t layer_stride;
} qcf_chunk_file;
size_t qcf_storage_staging_bytes(const qcf_dims* dims, const qcf_request* r);
qcf_status qcf_request_prefill_storage(const qcf_model* m, const qcf_request* r, const qcf_chunk_file* files,
                                       void* staging, size_t staging_bytes, const qcf_outputs* out, void* ws,
                                       size_t ws_bytes, void* compute_stream, void* copy_stream);
qcf_status qcf_storage_status(int* err);

/* Several requests whose retrieved chunks overlap (QCFuse 1: retrieved context chunks of
 * different queries overlap by more than 70 %; 2.B: a position-independent cache index
 * with content-based hash search).  A chunk is the same chunk when two requests pass the
 * same host K and V arrays with the same length (a content-keyed chunk store gives equal
 * chunks the same arrays).  On copy_stream every distinct chunk's K and V of a layer
 * cross the host link once, into a shared staging area, and are written from there into
 * each request's fused cache with that request's own offset (keys re-rotated, values
 * copied).  On compute_stream, consecutive requests with the same critical layer
 * (critical-layer selector, head dim 128, at most 128 query rows together once each
 * request's are rounded up to the attention row block) run their probe as one: each
 * probe layer's weights stream once for the group, each request attending only to its
 * own anchors and query rows; then every request runs its profile, selection and
 * recompute as qcf_request_prefill would, waiting only for the layers it reaches.
 * Results are bitwise those of qcf_request_prefill per request.
 *   reqs, outs   host arrays [n_req], 1 <= n_req <= 64, any selectors
 *   ws           device, qcf_batch_workspace_size(dims, reqs, n_req) bytes, caller-owned
 *   h2d_bytes    host, nullable: bytes this call sends host -> device
 * Enqueues only; argument errors are returned before any launch. */
size_t qcf_batch_workspace_size(const qcf_dims* dims, const qcf_request* reqs, int n_req);
qcf_status qcf_batch_prefill(const qcf_model* m, const qcf_request* reqs, const qcf_outputs* outs, int n_req,
                             void* ws, size_t ws_bytes, void* compute_stream, void* copy_stream, int64_t* h2d_bytes);

/* Embedding rows as fp32 residual: x[i] = embed[ids[rows[i]]] (device). */
qcf_status qcf_embed_rows(const qcf_model* m, const int32_t* ids, const int32_t* rows, int n, float* x,
                          void* stream);

/* Final RMSNorm of x_last (device fp32 [d]), logits = W_lm h (fp32 [vocab]),
 * first token = argmax, lowest index on ties.  ws: qcf_lm_head_workspace_size(). */
size_t qcf_lm_head_workspace_size(const qcf_dims* dims);
qcf_status qcf_lm_head(const qcf_model* m, const float* x_last, float* logits, int32_t* token, void* ws,
                       size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------ going on from a shared context
 *
 * What a program needs after the fused prefill, when several sequences (answers sampled
 * from one request, or several questions) go on from the same context: positions turned
 * into rotations for the layouts and scalings models use, a paged cache that grows with
 * each sequence, and the attention of such a batch, which reads the shared context for many
 * sequences at a time.  Tensors here are bf16 or fp16 (rotation also fp32); every tensor of
 * one call has the same type. */
#define QCF_BF16 0
#define QCF_F16 1
#define QCF_F32 2

/* Frequencies scaled for contexts longer than the model's original length.  Pair k of a
 * rotated width R has w_k = theta^(-2k/R); with s = factor, L0 = original:
 *   LINEAR  w_k / s
 *   BASE    theta replaced by theta * s^(R / (R - 2))                      (R > 2)
 *   TURNS   r = L0 w_k / (2 pi) turns over the original length, kept where r >= high,
 *           divided by s where r <= low, blended linearly in r between:
 *           w_k (g + (1 - g) / s), g = clamp((r - low) / (high - low), 0, 1)
 *   INDEX   the same blend, linear in the pair index between the indices that make `high`
 *           and `low` turns: i(t) = R ln(L0 / (2 pi t)) / (2 ln theta),
 *           a = max(0, floor(i(high))), b = min(R/2 - 1, ceil(i(low))),
 *           g = 1 - clamp((k - a) / max(b - a, 0.001), 0, 1)
 *           The blend ends at the last pair at the latest.  Methods that clamp b at R - 1 let it end
 *           behind that pair, and so have other rates wherever even the last pair makes more than
 *           `low` turns over L0 (theta 1e4, R 128, low 1: L0 above 54000; also small R).  Such rates,
 *           as any others, come in tables that the caller writes: a qcf_rope_table is only its
 *           cosines and sines.
 * amplitude multiplies cosine and sine (1 for none; a table used to move keys that are
 * already rotated wants 1). */
#define QCF_ROPE_SCALE_NONE 0
#define QCF_ROPE_SCALE_LINEAR 1
#define QCF_ROPE_SCALE_BASE 2
#define QCF_ROPE_SCALE_TURNS 3
#define QCF_ROPE_SCALE_INDEX 4
typedef struct qcf_rope_scaling {
  int kind;
  int original;   /* TURNS, INDEX: original context length, > 0 */
  double factor;  /* >= 1 */
  double low, high; /* TURNS: 0 <= low < high; INDEX: 0 < low < high */
  double amplitude;
} qcf_rope_scaling;

/* Fills device tables cos, sin [n_pos][R/2] fp32 with the angles of positions first_pos ..
 * first_pos + n_pos - 1: angles in fp64, values to 2^-44 and rounded once.  scaling NULL: none.  R even,
 * 2 <= R <= 512; 0 <= first_pos, first_pos + n_pos <= 2^31 - 1. */
qcf_status qcf_rope_table_fill(float* cos, float* sin, int first_pos, int n_pos, int R, double theta,
                               const qcf_rope_scaling* scaling, void* stream);

/* Rotates the first R = t->head_dim entries of every head and copies the others:
 * row i of x turns by the angles of position pos[i].
 *   x, y   device, rows of H heads of D contiguous entries; x_stride, y_stride entries
 *          from row to row (>= H D; multiples of 16 bytes are fastest).  y == x (same stride)
 *          rotates in place; any other overlap gives wrong rows.
 *   pos    device [n], each in [0, t->max_pos).  -1 marks a padding row: its row of y is
 *          left as it was.  Any other position outside the table does the same and sets
 *          QCF_DEV_BAD_INDEX.
 *   t      tables of rotated width R = head_dim, even, R <= D; D even, <= 512
 *   mode   QCF_ROPE_HALF pairs (k, k + R/2) or QCF_ROPE_INTERLEAVED pairs (2k, 2k + 1),
 *          | QCF_ROPE_INVERSE turns by the negative angle (undoes a rotation of amplitude
 *          1; also the gradient with respect to x)
 *   dtype  QCF_BF16, QCF_F16 or QCF_F32; arithmetic in fp32, rounded once.
 * One call takes n ceil(H / 4) (D / 2) / V < 2^32 - 256, V the largest of 8, 4, 2, 1 that divides
 * R / 2, (D - R) / 2 and both strides; more rows are refused (QCF_ERR_SHAPE) and go in several calls.
 * For bf16 and QCF_ROPE_HALF the bits are those of qcf_rope_reposition. */
#define QCF_ROPE_HALF 0
#define QCF_ROPE_INTERLEAVED 1
#define QCF_ROPE_INVERSE 2
qcf_status qcf_rope_apply(const void* x, int64_t x_stride, void* y, int64_t y_stride, int n, int H, int D, int dtype,
                          const int32_t* pos, const qcf_rope_table* t, int mode, void* stream);

/* A paged K/V cache: n_pages pages of page_size rows each, K and V laid out alike.  Row r of
 * head h of page p starts page_stride p + row_stride r + head_stride h entries from the base,
 * its D entries contiguous; strides are multiples of 16 bytes, so [page][row][head][D] and
 * [page][head][row][D] are both covered. */
typedef struct qcf_paged_kv {
  void* k;
  void* v;
  int dtype;               /* QCF_BF16 or QCF_F16 */
  int n_pages, page_size;  /* page_size a power of two, 8 .. 256 */
  int Hkv, D;              /* D 16, 64 or 128 */
  int64_t page_stride, row_stride, head_stride;
} qcf_paged_kv;

/* A batch of sequences over one shared prefix.  Rows of q and of new keys belong to sequence
 * b for row_start[b] <= row < row_start[b + 1]; they are its last tokens: row i of nq new rows
 * has own position kv_len[b] - nq + i and, for rotation, position prefix_len + that.  Rows in
 * no sequence (before the first, behind the last) are padding: without effect, whatever they
 * hold, their outputs left as they were.  Own token j of sequence b lives in page page_table[b][j / page_size], prefix
 * token j in page prefix_pages[j / page_size].
 * Lengths are read on the device, so that a captured graph can be replayed with others; the
 * host gives upper bounds.  A sequence that breaks one (or has fewer tokens than new rows,
 * or rows outside [0, n_rows)) is left out and sets QCF_DEV_BAD_INDEX. */
typedef struct qcf_paged_batch {
  int n_seq;                    /* <= 65535; attention: <= 2048 */
  int n_rows;                   /* rows of q, k_new, v_new, o, padding included */
  int max_q;                    /* bound on a sequence's new rows */
  int max_len;                  /* bound on kv_len, <= table_stride * page_size */
  const int32_t* row_start;     /* device [n_seq + 1], ascending */
  const int32_t* kv_len;        /* device [n_seq], own tokens with the new rows among them */
  const int32_t* page_table;    /* device [n_seq][table_stride] */
  int table_stride;
  int prefix_len;               /* 0: no prefix */
  const int32_t* prefix_pages;  /* device [ceil(prefix_len / page_size)], or NULL */
} qcf_paged_batch;

/* Writes the new keys and values of a batch into their pages, the keys rotated on the way,
 * and rotates the queries of the same rows in the same launch.
 *   k_new, v_new  device, rows of Hkv heads of D contiguous entries, kv_stride entries apart
 *   q, q_out      device, rows of Hq heads, q_stride and q_out_stride entries apart, or both
 *                 NULL; q_out == q (same stride) rotates in place
 *   t, mode       as in qcf_rope_apply (no QCF_ROPE_INVERSE); t NULL: nothing is rotated, keys
 *                 (and queries) are copied.  A row whose position is outside the table is left
 *                 out and sets QCF_DEV_BAD_INDEX, as is the K/V of a row whose page is outside
 *                 the cache (its q is still rotated).
 * Two rows of a batch never name the same cache slot (pages of different sequences differ). */
qcf_status qcf_paged_append(const qcf_paged_kv* cache, const qcf_paged_batch* batch, const void* k_new,
                            const void* v_new, int64_t kv_stride, const qcf_rope_table* t, int mode, const void* q,
                            int64_t q_stride, void* q_out, int64_t q_out_stride, int Hq, void* stream);

/* Attention of a batch over its shared prefix and its own tokens: for row i of sequence b at
 * own position p, o[i,h] = sum_j softmax_j(scale * q[i,h] . K_j) V_j over every prefix token
 * and own tokens j <= p, g = h / (Hq/Hkv), one softmax over both.
 * A KV head has Hq / Hkv score rows for each row of the batch.  A long prefix at head dim 64 or 128
 * is loaded once for every 2 floor(128 Hkv / Hq) rows of the batch (up to 256 score rows); a short
 * one, and any at head dim 16 or beside at most 16 score rows, once for every 16 of them.  What is loaded
 * again comes from L2 as far as it fits there.
 *   q    device, rows of Hq heads of D contiguous entries, q_stride entries apart
 *   o    device [n_rows][Hq][D], the cache's type; may be q itself (q_stride = Hq D), and
 *        overlaps nothing else
 *   lse  device [n_rows][Hq] fp32 natural-log sum of exp of the scaled logits, or NULL
 *   ws   device scratch of qcf_shared_prefix_attn_workspace_size() bytes; it needs no clearing;
 *        calls that overlap on the GPU (captured graphs replayed side by side among them) need
 *        separate scratch
 * scale > 0, Hq / Hkv <= 16, n_rows Hq < 2^24; bounds that allow more than about 2^31 tiles of 16
 * score rows and 32 keys are refused (QCF_ERR_SHAPE).  Cache rows behind a length (the rest of a last
 * page, pages not named) may hold anything, NaN included; a new token whose value holds NaN or infinity may spoil
 * every row of its own sequence.  A page outside the cache sets QCF_DEV_BAD_INDEX, and its
 * keys are left out of the softmax.  Products in the cache's type with fp32 sums, softmax in
 * fp32.  Results repeat bitwise for the same inputs and bounds.  Own tokens are loaded
 * again for every 16 score rows: meant for steps and questions.  New texts of hundreds of rows are right
 * but slow (4 of 1024 rows over 5120 keys, 32 heads over 8: 622 us, a third of the tensor rate). */
size_t qcf_shared_prefix_attn_workspace_size(const qcf_paged_kv* cache, const qcf_paged_batch* batch, int Hq);
qcf_status qcf_shared_prefix_attn(const qcf_paged_kv* cache, const qcf_paged_batch* batch, const void* q,
                                  int64_t q_stride, int Hq, float scale, void* o, float* lse, void* ws, size_t ws_bytes,
                                  void* stream);

/* ------------------------------------------------------------------ whole prompts and chunks of them
 *
 * Attention of many new tokens of a sequence at a time.  Both calls take head groups of
 * Hq / Hkv <= 128, read lengths on the device (a captured graph can be replayed with others
 * within the bounds) and share these arguments:
 *   q       device, rows of Hq heads of D contiguous entries, q_stride entries apart
 *   window  0: every key up to the row's own position; w > 0: the last w of them, its own among them
 *   o       device [n_rows][Hq][D], the type of q; may be q itself (q_stride = Hq D), and
 *           overlaps nothing else.  Rows in no sequence are left as they were
 *   lse     device [n_rows][Hq] fp32 natural-log sum of exp of the scaled logits, or NULL
 *   ws      device scratch of the matching *_workspace_size() bytes (0: ws may be NULL); it needs
 *           no clearing; calls that overlap on the GPU (captured graphs replayed side by side
 *           among them) need separate scratch
 * scale > 0; n_seq <= 8000; n_rows Hq < 2^24; bounds that allow more than about 2^27 key tiles of
 * 128 for 512 score rows each are refused (QCF_ERR_SHAPE).  Products in the type of q with fp32
 * sums, softmax in fp32.  Results repeat bitwise for the same inputs and bounds.  A NaN in a query
 * stays in its row and head; a key or value that holds NaN or infinity may spoil every row of its
 * own sequence (a prefix token: of the batch), masked or not, and no other. */

/* Causal attention of whole prompts packed one behind the other: rows row_start[b] <= row <
 * row_start[b + 1] are the tokens of sequence b in order, and token i attends to the tokens
 * j <= i of its own sequence (i - window < j with a window).
 *   k, v       device, rows of Hkv heads of D contiguous entries, kv_stride entries apart
 *   dtype      QCF_BF16 or QCF_F16
 *   row_start  device [n_seq + 1], ascending
 *   max_len    bound on a sequence's rows
 * D a multiple of 8, 8 .. 128 (computed as 64 or 128).  A sequence longer than max_len, or with
 * rows outside [0, n_rows), is left out and sets QCF_DEV_BAD_INDEX. */
size_t qcf_packed_causal_attn_workspace_size(int n_seq, int n_rows, int max_len, int Hq, int Hkv, int D);
qcf_status qcf_packed_causal_attn(const void* q, int64_t q_stride, const void* k, const void* v, int64_t kv_stride,
                                  int dtype, const int32_t* row_start, int n_seq, int n_rows, int max_len, int Hq,
                                  int Hkv, int D, float scale, int window, void* o, float* lse, void* ws,
                                  size_t ws_bytes, void* stream);

/* Attention of chunks of new tokens over a paged cache that holds them already
 * (qcf_paged_append): the arguments and the result of qcf_shared_prefix_attn, but for the window,
 * which counts positions (prefix_len + own).  Meant for chunks of prompts, alone or among the single
 * tokens of running sequences (4 of 1024 rows over 5120 keys, 32 heads over 8: 254 us, 622 by that call).  A
 * step of single tokens or short questions alone is faster there (64 single tokens over 5120 keys: 37 us, 56
 * here; questions of 33 to 64 rows over 16384: 99 and 106).  Cache rows
 * behind a length (the rest of a last page, pages not named) may hold anything, NaN included.  A page
 * outside the cache sets QCF_DEV_BAD_INDEX, and its keys are left out of the softmax; a row
 * left without any key gets o = 0 and lse = -infinity. */
size_t qcf_paged_chunk_attn_workspace_size(const qcf_paged_kv* cache, const qcf_paged_batch* batch, int Hq);
qcf_status qcf_paged_chunk_attn(const qcf_paged_kv* cache, const qcf_paged_batch* batch, const void* q, int64_t q_stride,
                                int Hq, float scale, int window, void* o, float* lse, void* ws, size_t ws_bytes,
                                void* stream);

/* ------------------------------------------------------------------ the pages of a cache
 *
 * Sequences whose tokens lie in pages, the same page ids in every layer's cache, with counts, tables
 * and lengths on the device (page_table and kv_len as qcf_paged_batch reads them; a shared prefix is
 * a sequence like any other, its row of the table the prefix_pages):
 *   refs        device [n_pages]: rows of the table that hold the page; 0: free
 *   page_table  device [n_seq][table_stride]; row b holds ceil(kv_len[b] / page_size) pages, what is
 *               behind them has no meaning and is left as it is
 *   kv_len      device [n_seq]
 * New pages are the lowest ids that were free before the call, in the order of its arguments:
 * pages given back by a call serve the next one.  A call does all it was asked or nothing: an
 * argument that its description rules out sets QCF_DEV_BAD_INDEX, too few free pages
 * QCF_DEV_NO_PAGES, and nothing has changed.  A page id outside the cache in a row that is only given
 * back or shared sets QCF_DEV_BAD_INDEX and is not counted.  Copies move whole entries; rows behind a length may hold anything.
 *   ws  device scratch of qcf_pages_workspace_size(pool, n) bytes; it needs no clearing; calls
 *       that overlap on the GPU need separate scratch (and may not share a pool)
 * n <= n_seq <= 65535, table_stride <= 2^20, 1 to 256 caches of one layout; refs 16-byte aligned,
 * the other tables 4. */
typedef struct qcf_page_pool {
  const qcf_paged_kv* caches;  /* HOST [n_caches]: every layer's */
  int n_caches;
  int32_t* refs;
  int32_t* page_table;
  int table_stride;
  int32_t* kv_len;
  int n_seq;
} qcf_page_pool;

/* Scratch of a call with n arguments (qcf_pages_compact: n = 0); 0 for a pool that is refused. */
size_t qcf_pages_workspace_size(const qcf_page_pool* pool, int n);

/* Sequence dst[i] goes on from src[i] for i < n (src, dst device [n]): what dst held is given back, it
 * takes the length of src, holds its full pages together with it, and has a copy of the page that src holds
 * in part.  Every dst once, and none of them a src; a src any number of times. */
qcf_status qcf_pages_fork(const qcf_page_pool* pool, const int32_t* src, const int32_t* dst, int n, void* ws,
                          size_t ws_bytes, void* stream);

/* Sequence seqs[i] (seqs NULL: i) gets the length new_len[i] for i < n, 0 <= new_len <= table_stride *
 * page_size (device [n]): pages behind it are given back, missing ones taken (their rows hold
 * anything).  Where the length changes and the last page that stays is held in part, and by others too,
 * its rows are copied to a new page, so that a later append writes into no other sequence.  Every
 * sequence once. */
qcf_status qcf_pages_resize(const qcf_page_pool* pool, const int32_t* seqs, const int32_t* new_len, int n, void* ws,
                            size_t ws_bytes, void* stream);

/* Moves the pages in use to the lowest ids: with *n_live (device) pages in use, the k-th of those at
 * or above n_live goes to the k-th free one below it, rows, counts and tables alike.  Every
 * holder of a page is a row of the table.  A length out of range: nothing has changed, and *n_live is -1.
 * Where pages move, a row's page that lies outside the cache, or at or above n_live without a count, sets
 * QCF_DEV_BAD_INDEX and stays in its row. */
qcf_status qcf_pages_compact(const qcf_page_pool* pool, int32_t* n_live, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* QCF_H_ */
