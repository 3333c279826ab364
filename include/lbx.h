/*
 * lbx.h -- C ABI of the tree-verify gated-DeltaNet library (GB300, sm_103a).
 *
 * The library computes the verify step of a hybrid model's gated-DeltaNet
 * (linear-attention) layers for a DDTree draft tree: the three tree-aware
 * state-rollback operations named in the Lucebox hub README (section
 * "02 DFlash DDtree", list "Implemented here": ggml_ssm_conv_tree,
 * ggml_gated_delta_net_tree, ggml_gated_delta_net_tree_persist), plus one
 * fused entry point that performs all three in a single pass.  DDTree itself
 * (same section, "Algorithms used") is a tree-structured verify: the draft is
 * a tree of B nodes given as a parent-index array, and every node is verified
 * against the state reached along its own root-to-node path.
 *
 * Notation.  L layers, Bq requests, N tree nodes (the budget), Hk key heads,
 * Hv value heads (Hv % Hk == 0; value head h reads key head h / (Hv/Hk)),
 * d = d_k = d_v, K conv width, C = 2*Hk*d + Hv*d conv channels ordered
 * q | k | v.  For each layer, request and value head h the recurrence is the
 * gated delta rule
 *     S_n = a_n S_p (I - b_n k_n k_n^T) + b_n v_n k_n^T,   o_n = q_scale * S_n q_n,
 * where p = parent[n] and S_p of the root (node 0) is the cached state of the
 * request's slot.  S is d_v x d_k, stored row-major [d_v][d_k].
 *
 * Conventions shared by every entry point:
 *   - Every array pointer is a DEVICE pointer owned by the caller; the
 *     library allocates nothing.  bf16 values are passed as their 16-bit
 *     patterns (uint16_t).  All arrays are dense and row-major in the index
 *     order written next to them; each must be 16-byte aligned.
 *   - Calls are asynchronous on `stream`.  The return value reports host-side
 *     argument checks and the launch: LBX_OK, LBX_EINVAL or LBX_ECUDA.
 *   - Structural errors that only the device can see (a parent array that is
 *     not a topologically numbered tree, a slot or accepted index out of
 *     range, two requests naming the same slot, a chain-mode input that is
 *     not a chain) are reported through `d_status` (an int32 in device memory,
 *     may be NULL): the kernel stores LBX_ETREE or LBX_EINVAL there and then
 *     writes NOTHING -- no outputs, no cache update.  `d_status` is never
 *     cleared by the library; zero it before the call to read it afterwards.
 *   - The draft tree: parent[b][0] == -1 (node 0 is the root, the last
 *     accepted token), and 0 <= parent[b][i] < i for i > 0.  One tree per
 *     request is shared by all layers.
 *   - Caches: state[L][n_slots][Hv][d][d] fp32 and conv_cache[L][n_slots][K-1][C]
 *     fp32 (raw pre-conv inputs, oldest row first; with K == 1 there is no
 *     conv cache and its pointer may be NULL).  Request b uses slot
 *     slot[b]; slots that no request names are never read or written.
 */
#ifndef LBX_H
#define LBX_H

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes. */
#define LBX_OK 0
#define LBX_EINVAL (-1) /* bad dimension, NULL pointer, size over a limit   */
#define LBX_ECUDA (-2)  /* a CUDA call or kernel launch failed               */
#define LBX_ETREE (-3)  /* invalid tree (device-detected, via d_status)      */
#define LBX_ETIMEOUT (-4) /* a bounded in-kernel wait gave up (via d_status) */
#define LBX_EPAGES (-5)  /* the page pool has too few free pages (via d_status) */

/* Limits. */
#define LBX_MAX_TREE_NODES 64 /* tree mode: N <= 64 nodes per request          */
#define LBX_CHAIN_CHUNK 64    /* chunked mode, CUDA-core path (d != 128): tokens
                                 per chunk; the d = 128 tensor-core chain kernel
                                 walks the chain 16 tokens at a time           */
#define LBX_MAX_CONV_WIDTH 4  /* 1 <= K <= 4                                    */
#define LBX_ACCEPT_MAX_NODES 4096 /* lbx_accept_walk: N <= 4096 nodes         */
#define LBX_DDTREE_MAX_K 8        /* lbx_ddtree_build: top-K, 1 <= K <= 8       */
#define LBX_DDTREE_MAX_DEPTH 64   /* lbx_ddtree_build: draft positions D <= 64  */
#define LBX_ATTN_HEAD_DIM 256     /* lbx_tree_attention: head dimension         */
#define LBX_EVICT_MAX_T (1 << 20) /* lbx_cache_evict: T <= 2^20 positions      */
#define LBX_ATTN_MAX_NODES 64     /* lbx_tree_attention and the operators of the
                                     bounded cache: N <= 64 tree nodes         */

/* Modes of lbx_verify_step. */
#define LBX_MODE_AUTO 0    /* tree if N <= LBX_MAX_TREE_NODES, else chunked     */
#define LBX_MODE_TREE 1    /* arbitrary tree, N <= LBX_MAX_TREE_NODES           */
#define LBX_MODE_CHUNKED 2 /* chain only (parent[i] == i-1), any N >= 1         */
#define LBX_MODE_TREE_CUDA_CORES 3 /* tree mode forced onto the CUDA-core kernel
                                      (same results; for cross-checking)       */

typedef struct lbx_cfg {
  int L;       /* gated-DeltaNet layers in the call (>= 1)                     */
  int Bq;      /* requests (>= 1)                                              */
  int N;       /* tree nodes per request (>= 1)                                */
  int Hk, Hv;  /* key / value heads, Hv % Hk == 0                              */
  int d;       /* head dimension d_k = d_v; 32 or 128                          */
  int K;       /* conv width, 1..LBX_MAX_CONV_WIDTH                            */
  int n_slots; /* cache slots in state / conv_cache (>= Bq)                    */
  float l2_eps;  /* q, k <- x / sqrt(sum x^2 + l2_eps); typical 1e-6           */
  float q_scale; /* o_n = q_scale * S_n q_n; 1.0 for the plain recurrence      */
  int mode;      /* LBX_MODE_*; used by lbx_verify_step only                   */
} lbx_cfg;

/* Human-readable text for a status code (static storage). */
const char *lbx_strerror(int status);

/* Bytes of workspace lbx_verify_step needs for cfg (0 on a bad cfg).  It
 * must be zero-filled once before its first use; two calls that run at the
 * same time must not share a workspace.  What it holds depends on the kernel
 * the configuration selects:
 *   - the tensor-core step (tree mode, d = 128, N <= 64): the per-request
 *     tree tables, per-(layer, request, key head) q/k operands (24 KB each
 *     at N <= 24, 64 KB at N <= 64) and per-(layer, request, value head)
 *     T/W records (2.8 KB at N <= 24, 17 KB at N <= 64) that its prep kernel
 *     writes and its step kernel reads, rewritten by every call;
 *   - the CUDA-core kernels: one arrival counter per (layer, request, key
 *     head); every call that runs to completion leaves them zero again. */
size_t lbx_workspace_size(const lbx_cfg *cfg);

/*
 * Tree conv (ggml_ssm_conv_tree; Lucebox hub README, "02 DFlash DDtree").
 * For node n and channel c:
 *     y = sum_{j=0}^{K-1} conv_w[l][c][K-1-j] * xhat_j[c],   out = y * sigmoid(y)
 * where xhat_0 is node n's input, xhat_1 its parent's, and so on up the
 * ancestor path; past the root the window continues into the slot's conv
 * cache, most recent cached row first.  Then q and k are L2-normalised per
 * key head over d channels (v is not).
 *   x          [L][Bq][N][C]   bf16   raw inputs of the tree nodes
 *   conv_w     [L][C][K]       bf16   depthwise conv weights, no bias
 *   conv_cache [L][n_slots][K-1][C] fp32 (read only here)
 *   parent     [Bq][N] int32, slot [Bq] int32
 *   qkv_out    [L][Bq][N][C]   fp32   (q scaled by nothing; q_scale is applied
 *                                      by lbx_tree_deltanet)
 * Requires cfg->N <= LBX_MAX_TREE_NODES.
 */
int lbx_tree_conv(const lbx_cfg *cfg, const uint16_t *x, const uint16_t *conv_w,
                  const float *conv_cache, const int32_t *parent, const int32_t *slot,
                  float *qkv_out, int32_t *d_status, cudaStream_t stream);

/*
 * Tree gated delta-rule recurrence (ggml_gated_delta_net_tree; same page).
 * Every node's state is the recurrence along its root-to-node path, started
 * from state[l][slot[b]][h]; o_n = q_scale * S_n q_n.
 *   qkv         [L][Bq][N][C]          fp32 (output of lbx_tree_conv)
 *   a, b        [L][Bq][N][Hv]         bf16 gates, already activated
 *   state       [L][n_slots][Hv][d][d] fp32 (read only here)
 *   parent      [Bq][N], slot [Bq]     int32
 *   o           [L][Bq][N][Hv][d]      fp32
 *   node_states [L][Bq][N][Hv][d][d]   fp32 per-node snapshots for a later
 *                                      lbx_tree_persist; may be NULL
 * Requires cfg->N <= LBX_MAX_TREE_NODES.
 */
int lbx_tree_deltanet(const lbx_cfg *cfg, const float *qkv, const uint16_t *a, const uint16_t *b,
                      const float *state, const int32_t *parent, const int32_t *slot, float *o,
                      float *node_states, int32_t *d_status, cudaStream_t stream);

/*
 * Persist (ggml_gated_delta_net_tree_persist; same page, "state rollback").
 * For each layer l and request b, with acc = accepted[b]:
 *   state[l][slot[b]]      <- node_states[l][b][acc]          (all Hv heads)
 *   conv_cache[l][slot[b]] <- the last K-1 entries of
 *                             [old cache rows, x of the path root..acc]
 * Both caches are updated in place.  The conv part copies bf16-exact values
 * and is bit-exact.
 *   x           [L][Bq][N][C] bf16, node_states [L][Bq][N][Hv][d][d] fp32,
 *   parent [Bq][N], slot [Bq], accepted [Bq] int32.
 */
int lbx_tree_persist(const lbx_cfg *cfg, const uint16_t *x, const float *node_states,
                     const int32_t *parent, const int32_t *slot, const int32_t *accepted,
                     float *state, float *conv_cache, int32_t *d_status, cudaStream_t stream);

/*
 * Fused verify step: tree conv + tree recurrence + persist in one pass.  The
 * cached state is read once, per-node states are never materialised, o is
 * written for every node, and only the accepted node's state and conv window
 * are written back (in place) to each request's slot.
 *   x [L][Bq][N][C], conv_w [L][C][K], a, b [L][Bq][N][Hv]   bf16
 *   parent [Bq][N], slot [Bq], accepted [Bq]                 int32
 *   state [L][n_slots][Hv][d][d], conv_cache [L][n_slots][K-1][C]  fp32, in/out
 *   o [L][Bq][N][Hv][d]                                     fp32, out
 *   workspace / workspace_bytes: >= lbx_workspace_size(cfg) bytes (see there)
 * Modes: in tree mode N <= LBX_MAX_TREE_NODES (the tensor-core step keeps node
 * labels as bytes, two nodes per lane of the warp that builds a request's
 * tables, and the CUDA-core step's S0 [K|Q] product tile covers at most 2N =
 * 128 columns at d = 128); chunked mode takes a chain of any length: at d =
 * 128 on the tensor cores in chunks of 16 tokens, otherwise on CUDA cores in
 * chunks of LBX_CHAIN_CHUNK tokens.  Distinct requests must name distinct
 * slots.
 */
int lbx_verify_step(const lbx_cfg *cfg, const uint16_t *x, const uint16_t *conv_w,
                    const uint16_t *a, const uint16_t *b, const int32_t *parent,
                    const int32_t *slot, const int32_t *accepted, float *state, float *conv_cache,
                    float *o, void *workspace, size_t workspace_bytes, int32_t *d_status,
                    cudaStream_t stream);

/* Capacity of lbx_verify_step_noalloc: L * Bq * Hk <= LBX_NOALLOC_MAX_GROUPS
 * arrival counters (256 KB). */
#define LBX_NOALLOC_MAX_GROUPS 65536

/*
 * lbx_verify_step without a workspace, for callers that cannot allocate
 * device memory -- for instance an engine that reserves all device memory
 * for its caches up front and allows no later cudaMalloc (which would also
 * synchronise the device), or a plugin inside a host framework that owns the
 * only allocator.  It computes exactly what lbx_verify_step computes; the
 * Lucebox hub README describes no such variant, so it has no passage of its
 * own to cite.
 *
 * Arguments and results are those of lbx_verify_step minus the workspace.
 * The arrival counters live in a fixed device array inside the library
 * (LBX_NOALLOC_MAX_GROUPS counters, 256 KB), which every GPU that loads the
 * library keeps until the process exits.  Configurations with
 * L * Bq * Hk > LBX_NOALLOC_MAX_GROUPS are rejected with LBX_EINVAL.  Where
 * lbx_verify_step would run the tensor-core step, whose workspace is larger
 * than the array, this function runs the CUDA-core tree kernel instead
 * (results agree within the tolerances of the tests; only speed differs).
 * The function allocates nothing: no cudaMalloc, cudaFree or other
 * allocating call.
 *   - The first call on each device looks up the array's device address
 *     (cudaGetSymbolAddress) with that device current, and may be the moment
 *     the library's kernels and the array are loaded onto that device; make
 *     that first call during set-up, before any stream capture.  The address
 *     is kept for the life of the process: it does not survive
 *     cudaDeviceReset (or any other teardown of the device's primary
 *     context), after which this entry point must not be called again.
 *   - Each call clears the counters it uses (cudaMemsetAsync on `stream`)
 *     before launching, since the array keeps the previous call's contents.
 *   - All calls on a device share the one array: calls that overlap on the
 *     GPU (other streams, other host threads) race on it.  Serialise them.
 */
int lbx_verify_step_noalloc(const lbx_cfg *cfg, const uint16_t *x, const uint16_t *conv_w,
                            const uint16_t *a, const uint16_t *b, const int32_t *parent,
                            const int32_t *slot, const int32_t *accepted, float *state,
                            float *conv_cache, float *o, int32_t *d_status, cudaStream_t stream);

/* Bytes of workspace lbx_accept_walk needs (0 on bad sizes).  It must be
 * zero-filled once before its first use (it holds one arrival counter per
 * request, which every call that runs to completion leaves at zero, and the
 * per-slice partial results); two calls that run at the same time must not
 * share it. */
size_t lbx_accept_workspace_size(int Bq, int N, int V);

/*
 * Verify argmax and greedy acceptance walk, on the device (Lucebox hub README,
 * "GPU draft top-K & verify-argmax (DFlash)": the target's per-node argmax is
 * taken from the logits buffer in place, so no vocabulary x nodes copy goes to
 * the host; greedy decoding, per the same README's serving notes, is the
 * high-acceptance mode).  Its accepted[] output feeds lbx_verify_step /
 * lbx_tree_persist directly, with no host round trip.
 *   logits [Bq][N][V] fp32 (4-byte aligned): the target's scores after each
 *     node (row n = the distribution of the token that follows node n);
 *   draft [Bq][N] int32: the draft token each node carries (node 0, the
 *     root = the last accepted token, is not read); parent [Bq][N] int32 as
 *     for lbx_verify_step (parent[0] = -1, parent[i] in [0, i));
 *   argmax_out [Bq][N] int32 (may be NULL): the target's choice at each node,
 *     the index of the largest logit, NaN ranking below every number, the
 *     lowest index among equal values (and in an all-NaN row);
 *   accepted_out [Bq] int32: the node where the walk stops -- from the root,
 *     repeatedly step to the lowest-index child whose draft token equals the
 *     target's choice at the current node;
 *   next_out [Bq] int32: the target's choice at the accepted node (the token
 *     that follows the accepted path).
 * All pointers are device pointers owned by the caller; the call is
 * asynchronous on `stream`.  Returns LBX_EINVAL for bad sizes (N >
 * LBX_ACCEPT_MAX_NODES), NULL or misaligned pointers or a short workspace,
 * LBX_ECUDA if the launch fails.  A request whose parent array breaks the
 * tree rules stores LBX_ETREE in *d_status (if not NULL) and writes none of
 * its outputs.  Draft tokens outside [0, V) never match.
 */
int lbx_accept_walk(int Bq, int N, int V, const float *logits, const int32_t *draft,
                    const int32_t *parent, int32_t *argmax_out, int32_t *accepted_out,
                    int32_t *next_out, void *workspace, size_t workspace_bytes,
                    int32_t *d_status, cudaStream_t stream);

/*
 * DDTree construction from the draft's top-K scores, on the device (Lucebox
 * hub README: DDTree, the tree-structured verify that beats chain verify at
 * the same budget, in "Algorithms used"; budget 22 on the RTX 3090 in
 * "Implemented here"; the draft's per-position top-K tokens, K in 1..8, in
 * "GPU draft top-K & verify-argmax (DFlash)").  The output parent array is
 * topologically numbered and feeds lbx_verify_step as is.
 *   logp [Bq][D][K] fp32: log-probabilities of the draft's top-K tokens at
 *     each of the D positions after the root (any order within a position;
 *     -inf allowed, NaN not);
 *   tok [Bq][D][K] int32: those tokens; root_tok [Bq] int32: the root's
 *     token (the last accepted token);
 *   parent_out, token_out [Bq][B] int32; depth_out [Bq][B] int32 and
 *     score_out [Bq][B] fp32 may be NULL; n_nodes_out [Bq] int32.
 * A node's score is the sum of the log-probabilities on its path, added in
 * fp32 from the root down; the tree is built best first: from the root
 * (score 0) the not-yet-added child of an added node with the highest score
 * joins next -- ties: the lower parent index, then the lower k -- until B
 * nodes or no candidate is left (n_nodes < B only when the whole trie of
 * depth D has fewer nodes).  Nodes are numbered in joining order; unused
 * slots get parent, token and depth -1 and score 0.  Device pointers owned
 * by the caller; asynchronous on `stream`.  Returns LBX_EINVAL for sizes
 * outside 1 <= B <= LBX_MAX_TREE_NODES, 1 <= K <= LBX_DDTREE_MAX_K,
 * 0 <= D <= LBX_DDTREE_MAX_DEPTH or NULL / misaligned pointers, LBX_ECUDA
 * if the launch fails.
 */
int lbx_ddtree_build(int Bq, int D, int K, int B, const float *logp, const int32_t *tok,
                     const int32_t *root_tok, int32_t *parent_out, int32_t *token_out,
                     int32_t *depth_out, float *score_out, int32_t *n_nodes_out,
                     cudaStream_t stream);

/* Bytes of workspace lbx_tree_attention needs for these shapes (0 if they
 * are not supported).  It must be zero-filled once before its first use;
 * every call that runs to completion leaves its counters at zero again; two
 * calls that run at the same time must not share a workspace. */
size_t lbx_attn_workspace_size(int L, int Bq, int N, int Hq, int Hkv, int dh, int T);

/*
 * Tree-masked attention of the hybrid target's full-attention layers in the
 * verify forward (Lucebox hub README: DDTree verifies the whole draft tree in
 * one target forward, "Algorithms used"; the full-attention layers keep a KV
 * cache, "--max-ctx N", and attend to all of it by default, "--fa-window N"
 * = 0).  Draft node n sits one position after its parent, so its query sees
 * the request's cached context and the tree nodes on its own root path
 * (its ancestors and itself):
 *     o[l][b][n][hq] = sum_j softmax_j(scale * q[l][b][n][hq] . k_j) v_j,
 * over j in { cache positions 0 .. ctx_len[b]-1 } u { tree nodes on the path
 * root -> n }, with KV head g = hq / (Hq/Hkv) (contiguous GQA groups).
 * Layers are a batch dimension sharing the tree and the context lengths.
 *   q        [L][Bq][N][Hq][dh]   bf16
 *   k_cache, v_cache [L][Bq][T][Hkv][dh] bf16 (T = capacity; may be NULL
 *            when T == 0); positions at or past ctx_len[b] are never used
 *   k_tree, v_tree   [L][Bq][N][Hkv][dh] bf16: the tree nodes' own keys and
 *            values (already projected and position-encoded by the caller)
 *   ctx_len  [Bq] int32 in 0..T;  parent [Bq][N] int32 (the draft tree)
 *   o        [L][Bq][N][Hq][dh]   fp32 out
 *   scale    > 0, finite (1/sqrt(dh) for plain scaled dot-product attention)
 * dh must be LBX_ATTN_HEAD_DIM and 1 <= N <= LBX_ATTN_MAX_NODES; Hq % Hkv ==
 * 0.  Computed on the tensor cores: S = Q K^T per key block and O += P V with
 * bf16 operands (P split into hi + lo) and fp32 accumulation, softmax in
 * fp32.  Device pointers owned by the caller (bf16 arrays and o 16-byte
 * aligned); asynchronous on `stream`.  Returns LBX_EINVAL for unsupported
 * shapes, NULL or misaligned pointers or a short workspace, LBX_ECUDA if the
 * launch fails; an invalid tree or a ctx_len outside 0..T is reported as
 * LBX_ETREE through d_status (nullable) and nothing is written.
 */
int lbx_tree_attention(int L, int Bq, int N, int Hq, int Hkv, int dh, int T, float scale,
                       const int32_t *ctx_len, const int32_t *parent, const uint16_t *q,
                       const uint16_t *k_cache, const uint16_t *v_cache, const uint16_t *k_tree,
                       const uint16_t *v_tree, float *o, void *workspace, size_t workspace_bytes,
                       int32_t *d_status, cudaStream_t stream);

/*
 * ---- The bounded, shared KV cache of the full-attention layers -------------
 *
 * Four operators for serving with a cache that does not grow without end and
 * prompts that requests share.  They take the draft tree of a verify step;
 * with N = 1 they are the plain decode step of one token.  lbx_window_attention
 * and lbx_prefix_attention give the attention output and the log-sum-exp of
 * each query; lbx_attention_mass turns the latter into per-key sums of
 * attention weights; lbx_cache_evict appends the accepted nodes' keys and
 * values to the cache and keeps the entries with the largest sums.
 * Layers are a batch dimension, as in lbx_tree_attention.  Notation: G =
 * Hq / Hkv query heads read one KV head (hq reads hq / G); depth(n) is node
 * n's distance from the root, whose query stands at position ctx_len[b]; the
 * accepted path is the nodes from the root to accepted[b].
 */

/* Element types of q, the keys, the values and o (16 bits each, passed as
 * their patterns). */
#define LBX_BF16 0
#define LBX_F16 1

typedef struct lbx_attn_cfg {
  int L, Bq, N;  /* layers, requests, tree nodes (1 <= N <= LBX_ATTN_MAX_NODES) */
  int Hq, Hkv;   /* query / KV heads, Hq % Hkv == 0                            */
  int dh;        /* head dimension: 64, 128 or 256                             */
  int T;         /* capacity of each request's cache (positions; may be 0)     */
  int P;         /* length of the shared prefix (lbx_prefix_attention only)    */
  int window;    /* a query sees the `window` positions up to its own (itself
                    included); 0 = all of them                                 */
  int n_sink;    /* the first n_sink positions stay visible / are never evicted */
  int dtype;     /* LBX_BF16 or LBX_F16                                        */
  float scale;   /* scale of q . k (> 0, finite)                               */
} lbx_attn_cfg;

/* Bytes of workspace lbx_window_attention (cfg->P == 0) or
 * lbx_prefix_attention (cfg->P > 0) needs (0 on a bad cfg).  It must be
 * zero-filled once before its first use (and after a call that reported
 * LBX_ETIMEOUT); every call that runs to completion leaves its counters at zero.
 * Calls of any configurations, of either function, may take turns on one
 * workspace that is large enough for each; two calls that run at the same time
 * must not share it. */
size_t lbx_cache_attn_workspace_size(const lbx_attn_cfg *cfg);

/*
 * Tree attention with a sliding window and a few first positions that stay
 * visible.  Cached position j < ctx_len[b] is visible to node n if
 *     window == 0  or  ctx_len[b] + depth(n) - j < window  or  j < n_sink,
 * and tree node m on n's root path (itself included) if the same holds for
 * m's position ctx_len[b] + depth(m).  A window counts places in the cache: it
 * needs one that holds every position in order, as an append-only cache does.
 * Where lbx_cache_evict has dropped entries, window must be 0 here and in
 * lbx_attention_mass.  Over the visible keys of each query
 *     o = sum_j exp(scale q.k_j - lse) v_j,  lse = log sum_j exp(scale q.k_j).
 *   q [L][Bq][N][Hq][dh], k_cache, v_cache [L][Bq][T][Hkv][dh] (may be NULL
 *   when T == 0), k_tree, v_tree [L][Bq][N][Hkv][dh], o [L][Bq][N][Hq][dh]
 *   out, all of cfg->dtype; lse [L][Bq][N][Hq] fp32 out, may be NULL;
 *   ctx_len [Bq] int32 in 0..T, parent [Bq][N] int32.
 * Keys and values of positions that no query of the request sees (at or past
 * ctx_len, before every window) may hold anything, NaN included.  A key that
 * one query of a request sees and another does not has to have a finite
 * value: it enters the other's sum with weight 0.  A query all of whose
 * scores are -inf gets o = 0 and lse = -inf; one with a NaN among its scores
 * gets NaN for both.
 * cfg->P must be 0.  Returns LBX_EINVAL for unsupported shapes, NULL or
 * misaligned pointers (16 bytes for the 16-bit arrays and the workspace, 4 for
 * the others) or a short workspace, LBX_ECUDA if a launch fails; an invalid
 * tree or a ctx_len outside 0..T stores LBX_ETREE in *d_status (may be NULL)
 * and writes nothing.
 */
int lbx_window_attention(const lbx_attn_cfg *cfg, const int32_t *ctx_len, const int32_t *parent,
                         const uint16_t *q, const uint16_t *k_cache, const uint16_t *v_cache,
                         const uint16_t *k_tree, const uint16_t *v_tree, uint16_t *o, float *lse,
                         void *workspace, size_t workspace_bytes, int32_t *d_status,
                         cudaStream_t stream);

/*
 * Attention of a batch whose requests share a prefix: every query sees the P
 * prefix positions, its request's ctx_len[b] cached positions and its root
 * path in the tree.  The prefix is held once for the batch and each layer's
 * is multiplied with the queries of all requests together.
 *   k_prefix, v_prefix [L][P][Hkv][dh]; the others as in lbx_window_attention
 * (o and lse are over all visible keys).  P >= 1; window and n_sink must be 0.
 */
int lbx_prefix_attention(const lbx_attn_cfg *cfg, const int32_t *ctx_len, const int32_t *parent,
                         const uint16_t *q, const uint16_t *k_prefix, const uint16_t *v_prefix,
                         const uint16_t *k_cache, const uint16_t *v_cache, const uint16_t *k_tree,
                         const uint16_t *v_tree, uint16_t *o, float *lse, void *workspace,
                         size_t workspace_bytes, int32_t *d_status, cudaStream_t stream);

/*
 * Attention weights per key, gathered over the queries of the accepted path:
 *     score[l][b][g][j]      += sum_{n on the path, hq / G = g} w(n, hq, j),
 *     score_tree[l][b][g][m]  = the same for tree node m on the path, else 0,
 * with w = exp(scale q.k - lse) for visible keys (visible as in
 * lbx_window_attention), else 0.  lse is what the attention call gave; with a
 * shared prefix it covers the prefix, whose keys are not scored; a query with
 * lse = -inf adds nothing; one with a NaN lse makes the sums of the keys it sees
 * NaN.
 *   accepted [Bq] int32 in 0..N-1; q, k_cache, k_tree, lse as above;
 *   score [L][Bq][Hkv][T] fp32, in/out (entries j >= ctx_len are not touched;
 *   may be NULL when T == 0); score_tree [L][Bq][Hkv][N] fp32 out.
 * cfg->P is not read.  Errors as in lbx_window_attention; an accepted index
 * out of range is reported like an invalid tree.
 */
int lbx_attention_mass(const lbx_attn_cfg *cfg, const int32_t *ctx_len, const int32_t *parent,
                       const int32_t *accepted, const uint16_t *q, const float *lse,
                       const uint16_t *k_cache, const uint16_t *k_tree, float *score,
                       float *score_tree, int32_t *d_status, cudaStream_t stream);

/*
 * Append the accepted path to the cache and keep at most `budget` entries per
 * (layer, request, KV head).  The candidates are the cached entries 0 ..
 * ctx_len[b]-1 and then the accepted path's nodes, root first; node n's
 * absolute position is seen[b] + depth(n).  With n candidates, size =
 * min(n, budget) stay: first those whose position is below n_sink or among
 * the last n_recent (>= seen_out[b] - n_recent), then by score, largest first
 * (NaN below every number, -0 equal to 0); ties go to the lowest index.
 * Cached entries that stay at an index below size do not move; the others
 * that stay, in order of their index, fill the free places below size, in
 * order.  Once entries have been dropped the order of those in the cache is
 * not that of their positions, which pos keeps; keys carry their position
 * encoding with them.  Until then (seen <= budget) the call appends in order.
 * Places at or past size keep what they held.
 *   k_cache, v_cache [L][Bq][T][Hkv][dh], score fp32 and pos int32
 *   [L][Bq][Hkv][T]: in/out; k_tree, v_tree [L][Bq][N][Hkv][dh], score_tree
 *   [L][Bq][Hkv][N]; ctx_len, seen, accepted [Bq], parent [Bq][N]: in;
 *   ctx_out [Bq] = size and seen_out [Bq] = seen + nodes of the path: out
 *   (LBX_EINVAL if they overlap each other, ctx_len, seen, parent or accepted;
 *   they are the next step's ctx_len and seen).
 * 1 <= budget <= T <= LBX_EVICT_MAX_T, n_sink >= 0, n_recent >= 0.  cfg->P, window and scale are
 * not read.  Errors as in lbx_attention_mass.
 */
int lbx_cache_evict(const lbx_attn_cfg *cfg, int budget, int n_recent, const int32_t *ctx_len,
                    const int32_t *seen, const int32_t *parent, const int32_t *accepted,
                    const uint16_t *k_tree, const uint16_t *v_tree, const float *score_tree,
                    uint16_t *k_cache, uint16_t *v_cache, float *score, int32_t *pos,
                    int32_t *ctx_out, int32_t *seen_out, int32_t *d_status, cudaStream_t stream);

/*
 * ---- The paged KV cache of the full-attention layers -----------------------
 *
 * Four operators for serving with a cache whose positions lie in pages of one
 * pool: lbx_page_tables gives the requests of a step the pages that their
 * lengths need, lbx_qk_norm_rope puts the new tokens' keys and values there,
 * lbx_paged_attention reads them, and lbx_page_commit keeps a verified path.
 * The new tokens of a batch are rows 0 .. start[Bq]-1 of M, request after
 * request (request b's are start[b] .. start[b+1]-1, any number of them, none
 * included); rows from start[Bq] on are padding: nothing is read from them and
 * what is written per row keeps what it held (slot and pos: -1).  Position p of
 * request b lies in page block_table[b][p / page] at p % page; of layer l's pool
 * [n_pages][page][Hkv][dh] that is row slot = block_table[b][p / page] * page +
 * p % page.  Layers are a batch dimension sharing lengths, tables and positions.
 */
#define LBX_PAGE_MAX_REQUESTS 2048
#define LBX_PAGED_MAX_GROUP 128 /* lbx_paged_attention: Hq / Hkv */

/* How lbx_paged_attention's softmax weights meet V, whose type has 16 bits.  SPLIT is as
 * accurate as lbx_window_attention in bf16 and takes longer: a tenth to a fifth for one layer
 * of draft trees or single tokens, up to two fifths for prompts and for many layers at
 * head dimension 256. */
#define LBX_WEIGHTS_ROUNDED 0 /* rounded once: 2^-8 of a weight in bf16, 2^-11 in f16 */
#define LBX_WEIGHTS_SPLIT 1   /* in two parts: 2^-16 and 2^-22                        */

typedef struct lbx_page_cfg {
  int L, Bq;      /* layers, requests (Bq <= LBX_PAGE_MAX_REQUESTS)             */
  int M;          /* rows of new tokens, padding included (>= 1)                */
  int Hq, Hkv;    /* query / KV heads, Hq % Hkv == 0, Hq * dh < 2^29            */
  int dh;         /* head dimension: 64, 128 or 256                             */
  int page;       /* positions per page: 16, 32, 64, 128 or 256                 */
  int n_pages;    /* pages of each layer's pool; L * n_pages * page < 2^31      */
  int max_pages;  /* columns of the block table; max_pages * page <= 2^30       */
  int dtype;      /* LBX_BF16 or LBX_F16                                        */
  float scale;    /* scale of q . k (> 0, finite)                               */
  int weights;    /* LBX_WEIGHTS_*: how softmax weights meet V                  */
} lbx_page_cfg;

/*
 * Block tables and slot maps of a step, from the requests' lengths.  Request b
 * has ctx_len[b] positions, gets new_len[b] more and holds its first held[b]
 * pages.  It leaves with exactly held_out[b] = ceil((ctx_len + new_len) / page):
 * the pages it holds beyond that go onto the free stack (request after request,
 * in order of position), then missing ones come off the stack's top (the same
 * order).  So an ended request (both lengths 0) gives its pages back, and one
 * whose draft was rejected those that only the draft had needed.  A page belongs to one
 * request: nothing counts references, and a page that two requests hold would go onto the
 * stack twice (lbx_prefix_attention reads a shared prompt from an array of its own).
 *   ctx_len, new_len, held [Bq], n_free [1] int32: in
 *   block_table [Bq][max_pages], free_list [n_pages] int32: in/out; entries past
 *     held_out, and places of the stack at or past its top, keep what they held
 *     or get what passed through them
 *   held_out [Bq], n_free_out [1] int32 out: the next step's held and n_free.
 *     They may not overlap the inputs (LBX_EINVAL)
 *   start [Bq + 1], slot [M], pos [M] int32 out
 * Of cfg, Bq, M, page, n_pages and max_pages matter.  Reported through d_status,
 * with nothing written: LBX_EPAGES if the pool has too few pages; LBX_EINVAL if a
 * length or count is negative, more tokens come than M, more pages are needed or
 * held than max_pages, or the stack would outgrow n_pages.  A page outside the pool
 * gives slot -1 for its positions, and LBX_EINVAL.  The call may be repeated
 * on the same inputs, with the same results.
 */
int lbx_page_tables(const lbx_page_cfg *cfg, const int32_t *ctx_len, const int32_t *new_len,
                    const int32_t *held, const int32_t *n_free, int32_t *block_table,
                    int32_t *free_list, int32_t *held_out, int32_t *n_free_out, int32_t *start,
                    int32_t *slot, int32_t *pos, int32_t *d_status, cudaStream_t stream);

/* How lbx_qk_norm_rope pairs the first `rot` dimensions of a head. */
#define LBX_ROPE_HALVES 0   /* pair i: dimensions i and i + rot/2 */
#define LBX_ROPE_ADJACENT 1 /* pair i: dimensions 2i and 2i + 1   */
#define LBX_ROPE_MAX_AXES 4

typedef struct lbx_rope_cfg {
  int rot;   /* dimensions that turn, even, 0 .. dh                              */
  int axes;  /* position axes, 1 .. LBX_ROPE_MAX_AXES                            */
  int section[LBX_ROPE_MAX_AXES]; /* pairs that turn with each axis, in order of the
                pairs; they add up to rot/2 (unused axes: 0)                     */
  int pairing; /* LBX_ROPE_*                                                     */
  float eps; /* of the norms (>= 0, finite)                                      */
} lbx_rope_cfg;

/*
 * Norms of queries and keys per head and their rotation by the tokens'
 * positions, in one pass that puts keys and values into their pages:
 *     y = x / sqrt(mean x^2 + eps) * weight       (x itself without a weight),
 *     (a, b) <- (a cos t - b sin t, b cos t + a sin t),  t = pos[axis(i)] inv_freq[i]
 * for every pair i of the first rot dimensions; values are copied.
 *   qkv [L][M][Hq + 2 Hkv][dh] of cfg->dtype: each row's query, key and value heads
 *   q_weight, k_weight [L][dh] fp32 (NULL: no norm)
 *   inv_freq [rot/2] fp32 (may be NULL when rot == 0; finite): any scaling of
 *     positions is in them.  Modulo a turn t is off by less than |pos| 2^-64 of a turn,
 *     then rounded to fp32: by 2^-24 of itself, 2^-26 of a turn at most
 *   pos [axes][M] int32, any values; slot [M] int32: a row's place in every layer's
 *     pool; a negative one marks a row that is skipped (padding)
 *   q_out [L][M][Hq][dh] out; k_pages, v_pages [L][n_pages][page][Hkv][dh]: the rows'
 *     slots are written, nothing else is touched
 * Sums and products are fp32, results rounded once.  A slot at or past
 * n_pages * page is reported as LBX_EINVAL through d_status and its row skipped.  Two
 * rows must not name one slot.  The outputs must not overlap the other arrays
 * (q_out and qkv: LBX_EINVAL).
 */
int lbx_qk_norm_rope(const lbx_page_cfg *cfg, const lbx_rope_cfg *rope, const uint16_t *qkv,
                     const float *q_weight, const float *k_weight, const float *inv_freq,
                     const int32_t *pos, const int32_t *slot, uint16_t *q_out, uint16_t *k_pages,
                     uint16_t *v_pages, int32_t *d_status, cudaStream_t stream);

/* Bytes of workspace lbx_paged_attention needs (0 on a bad cfg).  It must be
 * zero-filled once before its first use (and after a call that reported
 * LBX_ETIMEOUT); every call that runs to completion leaves its counters at zero.
 * Calls of any configurations may take turns on one workspace that is large
 * enough for each; two calls that run at the same time must not share it. */
size_t lbx_paged_workspace_size(const lbx_page_cfg *cfg);

/*
 * Attention of each request's new tokens over its pages.  Request b's tokens are at
 * positions ctx_len[b], ctx_len[b] + 1, .. of its cache, which holds their keys and
 * values already.  Token i sees the positions before ctx_len[b] and
 *     parent == NULL: its own and those of the tokens before it (a prompt's
 *                     chunk; with one token, the plain decode step);
 *     otherwise:      those of the tokens on its root path, itself included (a draft
 *                     tree, at most LBX_ATTN_MAX_NODES tokens per request):
 *                     parent[start[b]] == -1, 0 <= parent[start[b] + i] < i.
 *     o = sum_j exp(scale q.k_j - lse) v_j,  lse = log sum_j exp(scale q.k_j).
 *   start [Bq + 1], ctx_len [Bq], block_table [Bq][max_pages] int32; parent [M] int32
 *   or NULL; q [L][M][Hq][dh], k_pages, v_pages [L][n_pages][page][Hkv][dh] of
 *   cfg->dtype; o [L][M][Hq][dh] out of cfg->dtype, lse [L][M][Hq] fp32 out (may be
 *   NULL).
 * Sums and softmax statistics are fp32; the weights meet V in its type, as cfg->weights says
 * (at most 8 rows, tokens times Hq / Hkv, of every request over few keys: always in two parts,
 * which cost nothing there).
 * What a request's pages hold past its last token, and other pages, may be
 * anything, NaN included; a key that one query of a request sees and another
 * does not has to have a finite value; one that is not finite leaves that dimension of o
 * without a meaning (infinite or NaN).  A query all of whose scores are -inf gets o = 0
 * and lse = -inf; one with a NaN among its scores gets NaN for both.
 * M, padding included, and Bq decide how the work is laid out at head dimension 128: past 768
 * rows (tokens times Hq / Hkv) per request for long chunks, where single tokens over long caches
 * take 1.7 times as long.  A step of single tokens that is captured in a graph should have an
 * M of its own, not that of prompts.
 * Hq / Hkv <= LBX_PAGED_MAX_GROUP.  o, lse and the workspace must not overlap each other
 * or the inputs (each other or q: LBX_EINVAL).  Returns as lbx_window_attention.  Through
 * d_status, with nothing written: LBX_ETREE if start does not rise from 0 to at
 * most M, a length is negative or beyond the table, or a tree breaks its rules.  A
 * page outside the pool is not read: LBX_EINVAL through d_status, and the outputs of
 * that request hold nothing of use.
 */
int lbx_paged_attention(const lbx_page_cfg *cfg, const int32_t *start, const int32_t *ctx_len,
                        const int32_t *block_table, const int32_t *parent, const uint16_t *q,
                        const uint16_t *k_pages, const uint16_t *v_pages, uint16_t *o, float *lse,
                        void *workspace, size_t workspace_bytes, int32_t *d_status,
                        cudaStream_t stream);

/*
 * Keep the verified path of each request's draft tree: the keys and values of the
 * path's nodes, from the root to accepted[b], move to positions ctx_len[b],
 * ctx_len[b] + 1, .. (in place; a node's index is never below its depth), and
 * ctx_out[b] = ctx_len[b] + nodes of the path.  The positions behind hold what they
 * held.  A request without tokens keeps its length (accepted is not read).
 *   start, ctx_len, block_table, parent as in lbx_paged_attention (parent not
 *   NULL); accepted [Bq] int32, a node of the tree; k_pages, v_pages in/out;
 *   ctx_out [Bq] int32 out (LBX_EINVAL if it overlaps an int32 input).
 * Errors as in lbx_paged_attention; an accepted index out of range is reported
 * like an invalid tree, and a path through a page outside the pool does not move.
 */
int lbx_page_commit(const lbx_page_cfg *cfg, const int32_t *start, const int32_t *ctx_len,
                    const int32_t *block_table, const int32_t *parent, const int32_t *accepted,
                    uint16_t *k_pages, uint16_t *v_pages, int32_t *ctx_out, int32_t *d_status,
                    cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LBX_H */
