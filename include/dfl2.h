/*
 * dfl2: the DFlash 2 draft tail on one GB300 (sm_103a), as a C ABI.
 *
 * The tail runs once per draft-verify cycle, after the drafter's one-pass
 * forward and before the target's verify pass:
 *
 *   logits U [B,L,V] --top-16--> candidates --pair scores S_t(a,b)--> walk --> draft tokens
 *
 * plus the two-tap dynamic conv that the drafter applies before and after each
 * attention and feed-forward sublayer (5 layers x 4 insertion points).
 *
 * Sources (page title, section):
 *   [SEL]  "DFlash 2: Keep Drafting Parallel" (papercache.org digest of the
 *          Inco AI post), 方法细节 > 轻量级路径选择器 (Lightweight Path Selector):
 *          top-16 candidates per position, the pair-score equation
 *          S_t(a,b) = U_t(b) + <A(a) ⊙ H(h_t), B(b)>, and the walk over the
 *          precomputed scores starting from the last verified token.
 *   [CONV] same page, 方法细节 > 轻量级局部卷积 (Lightweight Local Convolution):
 *          Conv_k(x)_t = k_{t,0} ⊙ x_t + k_{t,1} ⊙ x_{t-1}, a learned base
 *          kernel plus a correction from the hidden state shared by every 16
 *          channels, and position 0 reading the last verified token.
 *   [TAB2] same page, Table 2 (+2.0M selector parameters) and the conv's
 *          "+16.5M" paragraph; these fix A(a) = W_A E[a], B(b) = W_B E[b],
 *          H(h) = sigmoid(W_H h) with W_* in R^{256 x d}, and a correction map
 *          of 2 d/16 rows for both taps.
 *   [WALK] "DFlash 2: The Drafter Stopped Guessing Alone" (rohitghumare.com),
 *          "Selection beats correction": greedy follows the best successor;
 *          sampling draws from the same scores.
 *
 * Conventions for every entry point:
 *   - Tensor pointers are DEVICE memory owned by the caller, row-major and
 *     contiguous, 16-byte aligned.  bf16 tensors are passed as uint16_t bit
 *     patterns.  Nothing is allocated by the library; scratch memory is a
 *     caller-provided workspace of at least *_workspace_size() bytes.
 *   - Work is enqueued on the caller's stream; no call synchronises the host
 *     (except dfl2_device_error, which says so).
 *   - Arguments are validated on the host before anything is launched; a bad
 *     argument returns a status and launches nothing.  Launch failures return
 *     DFL2_ERR_CUDA.  No call throws, aborts or prints.  dfl2_last_error()
 *     returns a thread-local message for the last failing call.
 *   - Fixed method sizes: k = 16 candidates, r = 256 selector rank; d must be a
 *     multiple of 16; V >= 16 (any V: logits rows need not start on 16 bytes),
 *     L >= 1, B >= 1.  The entry points of the NEXT rows keep narrower limits,
 *     stated at each (dfl2_verify: V % 4 == 0; dfl2_lmhead_topk: d % 8 == 0).
 *   - Every wait inside a kernel is bounded.  A wait that runs out (about 2 s
 *     of SM clock) records a code in a per-device error word
 *     (dfl2_device_error) and the kernel carries on without the data it
 *     waited for, so that launch's outputs are undefined; it still ends and
 *     leaves the context usable.  Once the error word holds such a code, every
 *     other wait that has lasted about 0.5 ms gives up too, so a launch whose
 *     pipeline stalls ends within a few seconds, not one full timeout per wait.
 *     (An index out of range, code 5, ends no wait, and a wait that runs out
 *     replaces it in the word.)
 *   - Workspaces must be zero-filled once before their first use (for example
 *     with dfl2_workspace_init); the library keeps them valid afterwards.
 *     Those of dfl2_tree_attn, dfl2_window_attn, dfl2_cache_weigh and
 *     dfl2_cache_evict are the exception: scratch of one call, which overwrites
 *     it, so it must not be a workspace that another entry point uses; calls that may
 *     run at the same time need one each.
 */
#ifndef DFL2_H
#define DFL2_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* A cudaStream_t (NULL = the legacy default stream). */
typedef struct CUstream_st* dfl2_stream;

typedef enum dfl2_status {
  DFL2_OK = 0,
  DFL2_ERR_INVALID_ARG = 1, /* null pointer, bad size, misaligned pointer, T < 0 ... */
  DFL2_ERR_UNSUPPORTED = 2, /* k != 16, r != 256, d or V not of a supported multiple */
  DFL2_ERR_WORKSPACE = 3,   /* workspace missing or smaller than *_workspace_size() */
  DFL2_ERR_CUDA = 4,        /* a CUDA runtime call or launch failed */
  DFL2_ERR_TIMEOUT = 5      /* a bounded in-kernel wait ran out (see dfl2_device_error) */
} dfl2_status;

typedef enum dfl2_dtype { DFL2_F32 = 0, DFL2_BF16 = 1, DFL2_F16 = 2 } dfl2_dtype;

/* Library version string, e.g. "dfl2 0.1 sm_103a". */
const char* dfl2_version(void);

/* Copies the calling thread's last error message (NUL-terminated, truncated to
 * len) and returns its full length. */
size_t dfl2_last_error(char* buf, size_t len);

/* Number of kernels this library has launched in this process (all devices). */
uint64_t dfl2_launch_count(void);

/* Engine of the projection GEMM (A = W_A E[a], B = W_B E[b], the gate's W_H h)
 * on its split-K path, the one that runs when the rows are few (batch 1 on the
 * drafter shapes: 241 + 256 gathered rows, 16 hidden rows); the batched path
 * always uses tcgen05.
 *   DFL2_PROJ_TENSOR (default): tcgen05 MMAs into a tensor-memory accumulator.
 *   DFL2_PROJ_WARP: the warp-level engine, each warp owning 32 output columns of
 *     its CTA's rows and computing them with mma.sync (m16n8k16, bf16 in, fp32
 *     accumulate) from the same shared-memory tiles.  It applies where a CTA
 *     holds 128 output columns (the batch-1 plans); elsewhere the tensor engine
 *     runs.
 * Process-wide (every device and thread), read when a call is enqueued; a
 * captured CUDA graph keeps the engine it was captured with.  Returns the
 * previous setting; an unknown value returns -1 and changes nothing. */
#define DFL2_PROJ_TENSOR 0
#define DFL2_PROJ_WARP 1
int dfl2_set_projection_engine(int engine);

/* Zero-fills a workspace on the stream (one cudaMemsetAsync). */
dfl2_status dfl2_workspace_init(void* ws, size_t ws_bytes, dfl2_stream stream);

/* Reads, and if clear != 0 resets, the current device's error word.  0 means no
 * kernel recorded a failed wait or an index out of range (5).  SYNCHRONISES the current device. */
dfl2_status dfl2_device_error(uint32_t* code, int clear);

/* ------------------------------------------------------------------ top-16
 * [SEL] "每个位置提取并保留 Top-16": for each of the B*L rows of logits [B,L,V]
 * (dtype float32 or bf16), the k = 16 largest logits, ordered by value
 * descending and then index ascending (-0.0 ties +0.0; NaN is not supported).
 * Writes cand_idx int32 [B,L,16] and cand_val float32 [B,L,16] (the logit,
 * widened exactly; a zero is written as +0.0).  ws: dfl2_topk_workspace_size
 * bytes (split-row partial lists and per-row tickets).
 */
size_t dfl2_topk_workspace_size(int B, int L, int V);
dfl2_status dfl2_topk(const void* logits, dfl2_dtype dtype, int B, int L, int V, int k,
                      int32_t* cand_idx, float* cand_val, void* ws, size_t ws_bytes,
                      dfl2_stream stream);

/* ------------------------------------------------------------------ LM head + top-16
 * The logits the top-16 step reads are the drafter's LM head applied to its
 * last hidden state ("DFlash 2: Keep Drafting Parallel", 方法细节 >
 * 轻量级路径选择器: U_t(.) is the drafter's own logit at position t).  This
 * entry point computes U_t(v) = sum_c hidden[t, c] * W_lm[v, c] (bf16 inputs,
 * float32 accumulation on the tensor cores) and keeps only the 16 largest per
 * row, inside the GEMM's epilogue: the [B*L, V] logits are never written.
 *   hidden  bf16 [B, L, d] row-major, device, 16-byte aligned.
 *   W_lm    bf16 [V, d] row-major, device, 16-byte aligned (a tied embedding
 *           table E may be passed).
 *   d       a multiple of 8 (16-byte rows); any V >= 16, any B*L >= 1.
 *   k       must be 16.
 *   Writes cand_idx int32 [B,L,16] and cand_val float32 [B,L,16] in the order
 *   of dfl2_topk (value descending, index ascending).  cand_val is the float32
 *   accumulator, so rows whose 16th and 17th logits differ by less than the
 *   accumulation error may pick either; with inputs whose partial sums are
 *   exact in float32 (e.g. small integers) the result equals dfl2_topk on the
 *   exact logits.  NaN/Inf inputs are not supported.
 *   ws: dfl2_lmhead_topk_workspace_size bytes (partial lists, not needing
 *   initialisation).  Two kernel launches on `stream`.
 * Errors: DFL2_ERR_INVALID_ARG (NULL/unaligned/host pointers, V < 16, B or L
 * < 1), DFL2_ERR_UNSUPPORTED (k != 16, d % 8 != 0), DFL2_ERR_WORKSPACE.
 */
size_t dfl2_lmhead_topk_workspace_size(int B, int L, int V, int d);
dfl2_status dfl2_lmhead_topk(const uint16_t* hidden, const uint16_t* W_lm, int B, int L, int V,
                             int d, int k, int32_t* cand_idx, float* cand_val, void* ws,
                             size_t ws_bytes, dfl2_stream stream);

/* ------------------------------------------------------------------ top-16, no allocation
 * No counterpart on the pages: a convenience of this library.  The same result
 * as dfl2_topk, for callers that cannot allocate device memory, such as serving
 * engines that reserve the GPU's memory for their own pool at start-up and
 * forbid later cudaMalloc, or plug-ins that get only input and output pointers.
 * The scratch dfl2_topk keeps in its workspace lives instead in a fixed 4 MiB
 * array of library-owned device memory (held on every GPU that loads the
 * library until the process exits); problems whose dfl2_topk_workspace_size
 * exceeds 4 MiB return DFL2_ERR_WORKSPACE without launching.  The first call on
 * a device looks up that array's address; make it before any stream capture.
 * All calls share the array, so calls whose kernels overlap on the GPU (other
 * streams or threads) race; calls in order on one stream are safe.
 */
dfl2_status dfl2_topk_noalloc(const void* logits, dfl2_dtype dtype, int B, int L, int V, int k,
                              int32_t* cand_idx, float* cand_val, dfl2_stream stream);

/* ------------------------------------------------------------------ pair scores
 * [SEL equation], [TAB2] reading:
 *   A(a) = W_A E[a], B(b) = W_B E[b], H(h_t) = sigmoid(W_H h_t)   (W_* [256,d], E [V,d])
 *   S[b,t,i,j] = cand_val[b,t,j] + sum_q A_q(a_i) H_q(h_{b,t}) B_q(cand_idx[b,t,j])
 * where a_i = cand_idx[b,t-1,i] for t >= 1, and for t = 0 only row i = 0 is
 * defined, with a_0 = verified_tok[b] (rows 1..15 of t = 0 are -inf).
 * hidden [B,L,d] bf16 is the drafter's final hidden state at each position.
 * scores float32 [B,L,16,16]; projections accumulate in float32.
 * ws: dfl2_select_workspace_size bytes (projected candidates and gates).
 */
size_t dfl2_select_workspace_size(int B, int L, int d);
dfl2_status dfl2_select(const int32_t* cand_idx, const float* cand_val,
                        const int32_t* verified_tok, const uint16_t* hidden, const uint16_t* E,
                        const uint16_t* W_A, const uint16_t* W_B, const uint16_t* W_H, int B,
                        int L, int V, int d, int r, float* scores, void* ws, size_t ws_bytes,
                        dfl2_stream stream);

/* ------------------------------------------------------------------ walk
 * [SEL "全并行打分与低延迟路径步进"], [WALK].  One sequential pass per
 * sequence over scores [B,L,16,16]: prev starts at row 0 of position 0 (the
 * verified token); at each t the step reads row prev of S[b,t] and picks
 *   temperature == 0: the lowest slot holding the row maximum (greedy);
 *   temperature  > 0: p_j = exp((S_j - max)/T), Z = sum_j p_j, u uniform in
 *                     [0,1), the first j with u Z < p_0 + ... + p_j.
 * u = (w >> 8) * 2^-24, w = word 0 of Philox4x32-10 (Salmon et al., SC'11)
 * with counter (t, lo32(cycle_offset), hi32(cycle_offset), 0) and key
 * (lo32(seeds[b]), hi32(seeds[b])).  Then prev = j*.
 * Writes tokens [B,L] = cand_idx[b,t,j*]; slots [B,L] = j* (nullable);
 * q [B,L,16] = p/Z, the draft distribution the verifier's rejection sampling
 * needs (one-hot when greedy; nullable).  seeds: device uint64 [B], may be NULL
 * when temperature == 0.
 */
dfl2_status dfl2_walk(const float* scores, const int32_t* cand_idx, int B, int L,
                      float temperature, const uint64_t* seeds, uint64_t cycle_offset,
                      int32_t* tokens, int32_t* slots, float* q, dfl2_stream stream);

/* ------------------------------------------------------------------ conv
 * [CONV equation], [TAB2] reading.  G = d/16 correction groups.
 *   corr[b,t,j,g] = sum_c W_c[j*G + g, c] x[b,t,c]          (j = tap 0, 1)
 *   k_j[c]        = base[j,c] + corr[b,t,j,c/16]
 *   y[b,t,c]      = k_0[c] x[b,t,c] + k_1[c] x[b,t-1,c],   x[b,-1,:] = x_prev[b,:]
 * x, y [B,L,d] bf16; x_prev [B,d] bf16 (the verified token's representation
 * at this insertion point); base float32 [2,d]; W_c bf16 [2G, d] with rows
 * [tap-0 groups; tap-1 groups].  float32 arithmetic, y rounded once to bf16
 * (nearest even).  y must not overlap x or x_prev.  No workspace.
 * base and W_c are weights: the call may read them before it waits for the
 * work queued ahead of it on `stream` (so that loading them overlaps that
 * work), hence no kernel still pending on `stream` may write them (set them,
 * e.g. with a copy, and let that copy complete or order it on another stream
 * that the caller synchronises, before the call).  x and x_prev are read only
 * after the earlier work on `stream` has finished.
 */
dfl2_status dfl2_conv2(const uint16_t* x, const uint16_t* x_prev, const float* base,
                       const uint16_t* W_c, int B, int L, int d, uint16_t* y,
                       dfl2_stream stream);

/* The same conv with a workspace.  With many positions (B*L > 64, d a multiple
 * of 64 and at least 512) the correction product is split over K across a
 * thread-block cluster and the partial products are exchanged through the
 * workspace, which lets the call spread over the whole GPU; otherwise the
 * call is the same as dfl2_conv2.  y is the same as dfl2_conv2's up to the
 * order of the float32 additions (each partial sum is added in a fixed
 * order, so a given shape always gives the same bits).
 * dfl2_conv2_workspace_size: bytes of device memory the call needs for this
 * shape on the current device (0: none, ws may be NULL); 0 also for an
 * unsupported shape or when no device is usable.
 * ws: device memory owned by the caller, at least that many bytes, not
 * overlapping x or y; its contents are scratch (no state is kept between
 * calls), and two calls that may run at the same time need separate
 * workspaces.  Errors: DFL2_ERR_WORKSPACE if ws is NULL or ws_bytes is too
 * small when bytes are needed; the argument errors of dfl2_conv2.
 */
size_t dfl2_conv2_workspace_size(int B, int L, int d);
dfl2_status dfl2_conv2_ws(const uint16_t* x, const uint16_t* x_prev, const float* base,
                          const uint16_t* W_c, int B, int L, int d, uint16_t* y, void* ws,
                          size_t ws_bytes, dfl2_stream stream);

/* ------------------------------------------------------------------ fused tail
 * top-16 -> pair scores -> walk in one call on one stream, with no host
 * synchronisation: the same results as dfl2_topk, dfl2_select and dfl2_walk
 * called in sequence.  cand_idx, cand_val, scores, slots and q are optional
 * outputs (NULL: kept in the workspace / not written).
 */
size_t dfl2_tail_workspace_size(int B, int L, int V, int d);
dfl2_status dfl2_tail(const void* logits, dfl2_dtype dtype, const int32_t* verified_tok,
                      const uint16_t* hidden, const uint16_t* E, const uint16_t* W_A,
                      const uint16_t* W_B, const uint16_t* W_H, int B, int L, int V, int d,
                      float temperature, const uint64_t* seeds, uint64_t cycle_offset,
                      int32_t* tokens, int32_t* slots, float* q, int32_t* cand_idx,
                      float* cand_val, float* scores, void* ws, size_t ws_bytes,
                      dfl2_stream stream);

/* ---------------------------------------------------------------------------
 * Precomputed token tables (a variant of the projections; the pages compute
 * A(a) = W_A E[a] and B(b) = W_B E[b] per candidate, "DFlash 2: Keep Drafting
 * Parallel", 方法细节 > 轻量级路径选择器, the definitions under the pair-score
 * equation).  Both maps are linear in E[.], so P_A = E W_A^T and P_B = E W_B^T,
 * built once per set of weights, give the same values per token (float32, the
 * accumulation order of the GEMM aside), and the per-cycle work shrinks to
 * gathering 1 KB rows instead of d-wide embedding rows.
 *
 * dfl2_tables_bytes(V): bytes of ONE table (float32 [V, 256]).
 * dfl2_tables_build: P_A, P_B (caller-owned device memory, dfl2_tables_bytes(V)
 *   each) from E [V, d] and W_A, W_B [256, d] (bf16, device).  d % 64 == 0.
 *   One tcgen05 GEMM launch; rebuild whenever E, W_A or W_B change.
 * dfl2_select_tables: as dfl2_select, with A(.) and B(.) read from the tables
 *   (E, W_A, W_B are not needed); the gate H = sigmoid(W_H h) is still computed
 *   per call.  Workspace: dfl2_select_workspace_size(B, L, d).
 * dfl2_tail_tables: as dfl2_tail with the tables.  The gate projection runs on
 *   a library-owned side stream (one per device and host thread), forked from
 *   and joined back to `stream` with events, beside the top-16; under CUDA
 *   graph capture the fork and join become graph edges.  Workspace:
 *   dfl2_tail_workspace_size(B, L, V, d).
 * Errors as for dfl2_select / dfl2_tail; a token outside [0, V) is recorded in
 * the device error word and read as row 0.
 * ------------------------------------------------------------------------- */
size_t dfl2_tables_bytes(int V);
dfl2_status dfl2_tables_build(const uint16_t* E, const uint16_t* W_A, const uint16_t* W_B, int V,
                              int d, float* P_A, float* P_B, dfl2_stream stream);
dfl2_status dfl2_select_tables(const int32_t* cand_idx, const float* cand_val,
                               const int32_t* verified_tok, const uint16_t* hidden,
                               const uint16_t* W_H, const float* P_A, const float* P_B, int B,
                               int L, int V, int d, int r, float* scores, void* ws,
                               size_t ws_bytes, dfl2_stream stream);
dfl2_status dfl2_tail_tables(const void* logits, dfl2_dtype dtype, const int32_t* verified_tok,
                             const uint16_t* hidden, const uint16_t* W_H, const float* P_A,
                             const float* P_B, int B, int L, int V, int d, float temperature,
                             const uint64_t* seeds, uint64_t cycle_offset, int32_t* tokens,
                             int32_t* slots, float* q, int32_t* cand_idx, float* cand_val,
                             float* scores, void* ws, size_t ws_bytes, dfl2_stream stream);

/* ---------------------------------------------------------------------------
 * dfl2_verify: verification of the drafted block against the target's
 * distributions, the step after the walk ("DFlash 2: Keep Drafting Parallel",
 * 方法细节 > 轻量级路径选择器, "全并行打分与低延迟路径步进": lossless rejection
 * sampling recovers the target's distribution; "DFlash 2: The Drafter Stopped
 * Guessing Alone", "One pass to draft, one pass to verify": the accepted prefix
 * is kept, the first miss is replaced by the target's own choice and the rest
 * dropped).  The sampling rule is the published speculative-sampling step
 * (Leviathan et al., ICML 2023; Chen et al., 2023).
 *
 *   p          [B, L+1, V] float32, device: the target's next-token
 *              probabilities; row t < L follows the verified token and the first
 *              t drafted tokens, row L follows the whole block.
 *   tokens     [B, L] int32: the drafted tokens (dfl2_walk / dfl2_tail).
 *   greedy     non-zero: keep tokens[t] while it is the lowest index holding the
 *              maximum of row t; the first miss is replaced by that index; when
 *              all L match, row L's argmax is appended.
 *              zero (sampling): with x = tokens[t] and q(x) = q[b,t,slots[t]],
 *              keep x iff u0 * q(x) < p_t(x); otherwise draw the replacement
 *              from max(0, p_t - q_t) (q_t is zero off cand_idx[b,t,:]): the
 *              first index, in order, whose running sum exceeds u1 * total (the
 *              last index with mass if rounding leaves none; p_t itself if the
 *              residual is zero).  When all L are kept, one token is drawn from
 *              row L the same way with u1.  u0, u1 = words 0 and 1 of
 *              Philox4x32-10 with counter (t, lo32(cycle), hi32(cycle), 1) and
 *              key = seeds[b], each (w >> 8) * 2^-24.
 *   slots, q, cand_idx, seeds: the walk's outputs [B,L], [B,L,16], the top-16
 *              candidates [B,L,16] and the per-sequence keys [B]; unused (may
 *              be NULL) when greedy.
 *   n_accepted [B] int32: drafted tokens kept (0..L).
 *   out_tokens [B, L+1] int32: the kept tokens, then the replacement or
 *              appended token, then -1.
 *   ws, ws_bytes: dfl2_verify_workspace_size(B, L, V) bytes of device memory
 *              (used by greedy; sampling may pass NULL and 0).
 * Constraints: L <= 128, 16 <= V <= 524288, V % 4 == 0.  Decisions are exact
 * (double precision); the replacement draw sums the row in single precision
 * within 512-element tiles and in double across tiles, so it can differ from
 * an exact sum only when u1 * total lies within rounding of a boundary.
 * Errors: DFL2_ERR_INVALID_ARG / UNSUPPORTED before any launch; a token or
 * slot out of range is recorded in the device error word (dfl2_device_error).
 * ------------------------------------------------------------------------- */
size_t dfl2_verify_workspace_size(int B, int L, int V);
dfl2_status dfl2_verify(const float* p, const int32_t* tokens, const int32_t* slots,
                        const float* q, const int32_t* cand_idx, int B, int L, int V, int greedy,
                        const uint64_t* seeds, uint64_t cycle_offset, int32_t* n_accepted,
                        int32_t* out_tokens, void* ws, size_t ws_bytes, dfl2_stream stream);

/* ---------------------------------------------------------------------------
 * The target's side of a draft-verify turn: a paged key/value cache, the
 * attention of a tree of drafted tokens over it, and the tree's acceptance.
 * No counterpart on the pages, which leave the target model out; a chain of L
 * drafted tokens (dfl2_tail) is the tree whose node i has parent i - 1.
 *
 * A turn of B sequences: node 0 of each tree is its last verified token, whose
 * keys and values are not in the cache yet; nodes 1 .. are drafted.
 *   dfl2_cache_reserve   pages for the nodes behind each sequence's length
 *   dfl2_tree_mask       parents -> which nodes each node sees
 *   per layer: dfl2_cache_write (the nodes' keys and values), dfl2_tree_attn
 *   dfl2_tree_accept     the target's choice at each node -> the kept path
 *   dfl2_cache_compact   the kept nodes' rows moved together, pages given back
 * dfl2_cache_fork and dfl2_cache_free begin and end sequences.  Layers with a window take
 * dfl2_window_attn, sampled trees dfl2_tree_verify; dfl2_cache_weigh and dfl2_cache_evict,
 * after the compaction, hold a sequence at a number of positions.
 *
 * The cache.  Element c of position `slot` in page `page`, key head h, layer l
 * of K is k[l*layer_stride + page*page_stride + h*head_stride +
 * slot*slot_stride + c] (strides in elements, any order of the dimensions);
 * V likewise from v.  The pages are shared by all layers and heads.
 *   dtype       DFL2_BF16, DFL2_F16 or DFL2_F32 (the attention: the first two).
 *   page_size   8, 16, 32, 64, 128 or 256 positions; head_dim * element size a
 *               multiple of 16 bytes, and so every stride; k, v 16-byte aligned.
 *   table       int32 [rows, cols]: entry i of a row is the page holding the
 *               sequence's positions i*page_size .., -1 where there is none.
 *   refs        int32 [pages]: how many table entries hold the page; 0 = free.
 *   free_bits   uint32 [ceil(pages/32)]: bit p%32 of word p/32 is set iff page
 *               p is free (bits past `pages` clear).
 * All of it is the caller's memory.  A new cache has table -1, refs 0 and every
 * page's bit set.  The calls below keep the three in step.  Pages are taken
 * lowest number first, in the order of the call's sequences and then of
 * positions, so the state after a call depends only on the state before it.
 * Lengths (how many positions of a sequence hold committed tokens) are the
 * caller's int32 arrays; no call needs them on the host.  Only the page that
 * holds position `length` and those behind it are ever written for a sequence,
 * and these are never shared: dfl2_cache_fork copies the partly filled one.
 *
 * Arguments that the calls share:
 *   table_rows  int32 [B], the table row of each sequence, distinct within a
 *               call; NULL: sequence b is row b.
 *   length      int32 [B]: committed positions of each sequence, 0 .. 2^30.
 *   count       int32 [B]: how many of the T nodes (or tokens) of the sequence
 *               there are, 0 .. T (other values are taken to the nearer end);
 *               NULL: T each.
 *   B           1 .. 65535 sequences; dfl2_cache_reserve and dfl2_cache_fork, which
 *               serve them in order, 1 .. 4096.
 *   integer arrays need 4-byte alignment, tensors of elements 16-byte.
 * A table row or page number out of range is recorded in the device error word
 * (dfl2_device_error); that sequence or position is then left out.  So is a
 * sequence whose length is out of range, except that dfl2_cache_reserve and
 * dfl2_cache_fork only report it unserved.
 * ------------------------------------------------------------------------- */
typedef struct dfl2_cache {
  void* k;
  void* v;
  int32_t dtype; /* dfl2_dtype */
  int32_t layers, pages, kv_heads, page_size, head_dim;
  int64_t layer_stride, page_stride, head_stride, slot_stride;
  int32_t* table;
  int32_t rows, cols;
  int32_t* refs;
  uint32_t* free_bits;
} dfl2_cache;

/* Pages for positions length .. length+count-1 of each sequence: the missing
 * entries of its table row in that range are filled.  served [B] int32: 1, or 0
 * where the free pages did not reach (sequences are served in order while they
 * do; one that needs no page is served in any case) or the row has too few
 * entries; such a sequence is left as it was.  1 <= B <= 4096, T >= 0, and B
 * times the entries that T positions may lie in (at most cols) below 2^31. */
dfl2_status dfl2_cache_reserve(const dfl2_cache* cache, int B, int T, const int32_t* table_rows,
                               const int32_t* length, const int32_t* count, int32_t* served,
                               dfl2_stream stream);

/* Rows of keys and values into layers layer .. layer+n_layers-1, positions
 * length .. length+count-1.  k_new, v_new: element c of head h, token t,
 * sequence b, layer layer+l at l*new_strides[0] + b*new_strides[1] +
 * t*new_strides[2] + h*new_strides[3] + c (host array of four element strides,
 * multiples of 16 bytes, for both).  Positions without a page are skipped and
 * recorded as out of range.  T >= 0 (0: k_new and v_new may be NULL). */
dfl2_status dfl2_cache_write(const dfl2_cache* cache, int layer, int n_layers, const void* k_new,
                             const void* v_new, const int64_t* new_strides, int B, int T,
                             const int32_t* table_rows, const int32_t* length,
                             const int32_t* count, dfl2_stream stream);

/* After acceptance: in every layer, the rows of nodes path[b,0..n_path-1] (as
 * dfl2_tree_accept gives them: strictly ascending) move to positions length,
 * length+1, ..; pages of the range length .. length+count-1 that hold none of
 * the kept rows are given back; new_length[b] = length[b] + n_path[b] (may be
 * the same array as length; a sequence left out keeps its length).  path int32 [B,T], n_path int32 [B] (0 drops all
 * drafted rows).  T <= 256. */
dfl2_status dfl2_cache_compact(const dfl2_cache* cache, int B, int T, const int32_t* table_rows,
                               const int32_t* length, const int32_t* count, const int32_t* path,
                               const int32_t* n_path, int32_t* new_length, dfl2_stream stream);

/* Sequence dst[i] (a table row whose entries are all -1) becomes a copy of the
 * first length[i] positions of table row src[i], for n pairs in order; the same
 * src may come several times, a dst once and as no src.  Whole pages are
 * shared; the positions of a partly filled last page are copied in every layer
 * into a page taken for it.  served [n] int32: 1, or 0 where the free pages did
 * not reach (in order, as in dfl2_cache_reserve), dst held pages already or src
 * lacks some; then dst is left as it was.  1 <= n <= 4096. */
dfl2_status dfl2_cache_fork(const dfl2_cache* cache, int n, const int32_t* src,
                            const int32_t* dst, const int32_t* length, int32_t* served,
                            dfl2_stream stream);

/* Gives back every page of n table rows and sets their entries to -1. */
dfl2_status dfl2_cache_free(const dfl2_cache* cache, int n, const int32_t* table_rows,
                            dfl2_stream stream);

/* A sequence longer than `keep` positions gives up those of least weight: its first
 * `sinks` and last `recent` positions stay, and of the others as many of the largest
 * weights as make `keep` (equal ones: the lower positions; NaN counts as -inf).  In every
 * layer the rows that stay move together, in order, to positions 0 .. keep-1, their weights
 * with them, and the pages that held only positions keep .. length-1 are given back (those
 * reserved past the length stay).  One no longer than `keep` stays as it is.
 * dfl2_cache_fork copies no weights: the caller copies the source's row of them before the
 * fork is weighed or evicted.
 *   weight      float32 [rows, cols*page_size]: of position j of table row r (as
 *               dfl2_cache_weigh leaves it); what lies behind the new length stays.
 *   kept        int32 [B,keep]: the old positions of the ones that stay, in order (for what
 *               else the caller keeps by position), then -1.
 *   new_length  int32 [B]: min(length, keep) (may be the same array as length).
 *   served      int32 [B]: 1, or 0 where a page of the sequence is missing, where one that
 *               would be written is shared with another sequence (dfl2_cache_fork), or where
 *               the sequence cannot be that long; it is then left as it was, with kept -1.
 *   ws          dfl2_cache_evict_workspace_size bytes of scratch (not zero-filled, and not
 *               shared with an entry point whose workspace holds counters).
 * 1 <= keep <= 2^30; sinks, recent >= 0, together at most keep.  Two kernel launches. */
size_t dfl2_cache_evict_workspace_size(int B, int keep);
dfl2_status dfl2_cache_evict(const dfl2_cache* cache, int B, const int32_t* table_rows,
                             const int32_t* length, int keep, int sinks, int recent, float* weight,
                             int32_t* kept, int32_t* new_length, int32_t* served, void* ws,
                             size_t ws_bytes, dfl2_stream stream);

/* parents int32 [B,T]: parents[b,i] < i is the node that node i follows, -1
 * none (node 0).  mask uint32 [B,T,ceil(T/32)]: bit j of row i is set iff j is i
 * or an ancestor of i.  depth int32 [B,T] (nullable): the number of ancestors.
 * Rows at and past count are 0.  A parent out of range is recorded and read as
 * -1.  1 <= T <= 256. */
dfl2_status dfl2_tree_mask(const int32_t* parents, int B, int T, const int32_t* count,
                           uint32_t* mask, int32_t* depth, dfl2_stream stream);

/* The path of the target's tokens through each tree.  tokens int32 [B,T] (that
 * of node 0 is not read), target int32 [B,T]: the target's token after node i.
 * From node 0 on: the lowest-numbered child whose token is the node's target
 * token, while there is one.  path int32 [B,T]: the nodes, node 0 first, then
 * -1; n_path int32 [B]; next_token int32 [B]: the last node's target token, the
 * next turn's node 0.  With greedy targets this is the target's own greedy
 * decoding; with target[b,i] drawn from the target's distribution at node i it
 * keeps that distribution.  count 0 gives n_path 0 and next_token -1.
 * 1 <= T <= 256. */
dfl2_status dfl2_tree_accept(const int32_t* tokens, const int32_t* parents,
                             const int32_t* target, int B, int T, const int32_t* count,
                             int32_t* path, int32_t* n_path, int32_t* next_token,
                             dfl2_stream stream);

/* The path of sampled tokens through each tree: speculative sampling with several
 * drafted tokens at a position (the step of dfl2_verify, Leviathan et al., ICML 2023;
 * Chen et al., 2023, applied to a node's children one after the other with what the
 * ones before left of the target's distribution).  The tokens of the path and
 * next_token follow the target's distribution, whatever q is, if the children of
 * node i were drawn from it.
 *   p           float32 [B,T,V]: the target's probabilities of the token after node i;
 *               each row is taken to sum to 1.
 *   tokens, parents  int32 [B,T] (node 0's token is not read; a parent that is not
 *               below its node makes the node no child).
 *   cand_idx, q int32 and float32 [B,T,16]: the children of node i were drawn from the
 *               candidates cand_idx[b,i] with weights q[b,i] (dfl2_walk's; they need
 *               not sum to 1, but to a finite number), in the order of their numbers.  A candidate named twice
 *               counts at its lowest slot; one outside [0, V) is recorded and, as a
 *               weight that is not above 0, counts as 0.
 *   replace     0: children drawn without replacement (distinct); else independently.
 *   u           float32 [B,T], uniform in [0,1): u[b,c] decides about node c >= 1,
 *               u[b,0] draws next_token.
 * From node 0 on: r = p[b,i], d = q[b,i].  For each child c of the node, x = its token:
 * passed over if d(x) = 0, else kept, and the next node, if u[b,c] d(x)/|d| < r(x)/|r|;
 * else r becomes max(0, r/|r| - d/|d|) and, without replacement, d(x) becomes 0; if r is
 * then 0 everywhere (p never exceeds q), it becomes p and the node's other children are
 * passed over.  When no child is kept: next_token = the first index, in order, at which
 * the running sum of r exceeds u[b,0] times its total (the last one with r > 0 if
 * rounding leaves none; of p if r sums to 0, -1 if that does too).
 * path, n_path, next_token: as dfl2_tree_accept's.  Decisions are taken in
 * arithmetic of about 46 bits; the running sums are off by at most 2^-37 + V 2^-61 of their
 * total.  Rows with NaN, Inf or values below 0 are not supported.
 * 1 <= T <= 256, 1 <= V <= 2^30; p, cand_idx 16-byte aligned (rows of p need not be). */
dfl2_status dfl2_tree_verify(const float* p, int B, int T, int V, const int32_t* tokens,
                             const int32_t* parents, const int32_t* count,
                             const int32_t* cand_idx, const float* q, const float* u, int replace,
                             int32_t* path, int32_t* n_path, int32_t* next_token,
                             dfl2_stream stream);

/* Attention of the nodes over the cache, in one layer:
 *   s_j = scale <q[b,i,h], K[b,j,h*kv_heads/q_heads]>
 *   out[b,i,h] = sum_j softmax(s)_j V[b,j]   over the positions j that node i
 * sees: all of 0 .. length-1 and, of the nodes at length .. length+count-1,
 * those whose bit is set in mask[b,i] (uint32 [B,T,ceil(T/32)]; NULL: node i
 * sees nodes 0 .. i, a chain).  What a position that a node does not see holds
 * has no influence on it, NaN included.  A node that sees nothing, or nothing
 * but scores of -inf, and rows at and past count have out = 0, lse = -inf.
 *   q, out      bf16 or fp16 as the cache; element c of head h, node i,
 *               sequence b at b*strides[0] + i*strides[1] + h*strides[2] + c
 *               (host arrays of three element strides, positive multiples of 8;
 *               that of a dimension of one entry is not read).  out must not
 *               overlap q or the cache.
 *   lse         float32 [B,T,q_heads] (nullable): log sum_j exp(s_j).
 *   head_dim 64, 128 or 256; q_heads a multiple of kv_heads, at most 128 times it;
 *   1 <= T <= 256; 1 <= B <= 65535; every cache stride of a dimension of more than
 *   one entry positive.
 *   ws          dfl2_tree_attn_workspace_size bytes, scratch only: need not be
 *               zero-filled, and is overwritten, so not shared with the other entry
 *               points, whose workspaces hold counters (zero-fill it again before).
 * Scores, softmax and sums are float32; the weights are rounded to the cache's
 * type for the product with V (fp16: times 2^7, so that weights down to 2^-21 of
 * a row's largest keep its 11 bits). */
size_t dfl2_tree_attn_workspace_size(int B, int T, int q_heads, int kv_heads, int head_dim,
                                     dfl2_dtype dtype);
dfl2_status dfl2_tree_attn(const void* q, const int64_t* q_strides, const dfl2_cache* cache,
                           int layer, int B, int T, int q_heads, const int32_t* table_rows,
                           const int32_t* length, const int32_t* count, const uint32_t* mask,
                           float scale, void* out, const int64_t* out_strides, float* lse,
                           void* ws, size_t ws_bytes, dfl2_stream stream);

/* The same in a layer whose tokens see a window and the first few positions (sinks): of
 * the positions that dfl2_tree_attn lets node i see, those at or past `sinks` only count
 * if they are less than `window` positions before it.  Node i stands at position
 * length + depth[b,i] (int32 [B,T], as dfl2_tree_mask gives it; other values than
 * 0 .. T-1 are taken to the nearer end; NULL: length + i, only without a mask), and so does
 * a node that it sees.  Only the sinks and what the first node's window reaches are read,
 * and pages that lie wholly between the two need not be there.
 *   sinks 0 .. 2^30; window 1 .. 2^30 (1: itself).
 * Positions are the cache's.  Behind dfl2_cache_evict, which takes some out of the middle, they
 * are the text's for this layer only if the eviction's `recent` is at least window - 1 and its
 * `sinks` at least these.
 * All else, the workspace included, as for dfl2_tree_attn. */
dfl2_status dfl2_window_attn(const void* q, const int64_t* q_strides, const dfl2_cache* cache,
                             int layer, int B, int T, int q_heads, const int32_t* table_rows,
                             const int32_t* length, const int32_t* count, const uint32_t* mask,
                             const int32_t* depth, int sinks, int window, float scale, void* out,
                             const int64_t* out_strides, float* lse, void* ws, size_t ws_bytes,
                             dfl2_stream stream);

/* What each position received of the attention of the tokens that a turn kept, added to its
 * weight (for dfl2_cache_evict): called for a layer without a window, after acceptance and
 * compaction, with the q and lse of that layer's attention call.
 *   weight[r,j] += sum over i, h of exp(scale <q[b,path[b,i],h], K[b,j]> - lse[b,path[b,i],h])
 * for the kept queries i = 0 .. n_path-1, which stand at positions length + i now, over the
 * positions j <= length + i that each sees; r is the sequence's table row.
 *   q           as for dfl2_tree_attn (strides: non-negative multiples of 8).
 *   lse         float32 [B,T,q_heads], as dfl2_tree_attn left it (not dfl2_window_attn, whose
 *               sums leave positions out that are counted here); a query and head whose lse
 *               is not finite adds nothing.
 *   length      int32 [B]: committed positions before this turn's.
 *   path        int32 [B,T]: node numbers (dfl2_tree_accept's); NULL: 0, 1, ..  One out of
 *               0 .. T-1 is recorded and left out.  n_path int32 [B], taken to 0 .. T;
 *               NULL: T.  So a prompt's chunk, or a token, needs neither.
 *   weight      float32 [rows, cols*page_size] (rows and cols: the table's).
 *   first       non-zero: the weights of positions length .. length+n_path-1 are set instead
 *               (the first layer's call of a turn).
 * A position without a page is recorded, and its weight left as it was; a sequence whose
 * positions its table row cannot hold is recorded and left out.
 * Shapes and types as for dfl2_tree_attn.  ws: dfl2_cache_weigh_workspace_size bytes of scratch
 * (not zero-filled, and not shared with an entry point whose workspace holds counters).
 * Each weight is a sum in a fixed order: the same call gives the same bits. */
size_t dfl2_cache_weigh_workspace_size(void);
dfl2_status dfl2_cache_weigh(const void* q, const int64_t* q_strides, const float* lse,
                             const dfl2_cache* cache, int layer, int B, int T, int q_heads,
                             const int32_t* table_rows, const int32_t* length, const int32_t* path,
                             const int32_t* n_path, float scale, int first, float* weight, void* ws,
                             size_t ws_bytes, dfl2_stream stream);

#ifdef __cplusplus
}
#endif
#endif /* DFL2_H */
