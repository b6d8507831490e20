/*
 * kda.h -- C ABI of the GB300 (sm_103a) Kimi Delta Attention forward library.
 *
 * The operation (K3 convention, state S in R^{d_k x d_v}):
 *   S_t = (I - beta_t k_t k_t^T) Diag(alpha_t) S_{t-1} + beta_t k_t v_t^T,
 *   o_t = S_t^T q_t,
 *   alpha_t = exp(g_t),  g_t = g_min * sigmoid(exp(A_h) * z_t)   (per channel)
 * ("Kimi K3 模型结构（7）：结构决定系统", section "KDA 上下文并行", eq. (1);
 *  "Kimi K3 模型结构（2）：序列维度（下），chunkwise 并行与下界衰减", section
 *  "K3 的改动：下界衰减", eq. (5); "Kimi K3: the Manos, the Mythos ..."
 *  (SemiAnalysis), section "FlashKDA 算法", delta form).
 * No query scaling is applied; beta is taken after its sigmoid and q, k are
 * taken already L2-normalised.
 *
 * Conventions shared by every entry point
 *   - Pointers marked (device) are device memory owned by the caller; the
 *     library never allocates or frees them and keeps no reference after the
 *     call returns.  Pointers marked (host) are read during the call only.
 *   - Every call is asynchronous on `stream` (a cudaStream_t; NULL = legacy
 *     default stream).  Results are ready when the stream reaches that point.
 *   - d_k = d_v = D must be 128 (KDA_ERR_UNSUPPORTED otherwise).
 *   - Layouts are row-major, innermost dimension last, no padding:
 *       q, k, z : [T_total, H, D]      v, o : [T_total, H, D]
 *       beta    : [T_total, H]         A    : [H]
 *       states  : [n_seqs, H, D(d_k), D(d_v)]  (fp32)
 *   - dtype selects the element type of q, k, v and o: KDA_BF16 or KDA_F32.
 *     z, A, beta and all states are always fp32.
 *   - Return value: KDA_OK or one of the KDA_ERR_* codes below.  Argument
 *     errors are detected on the host before anything is launched.  Checks
 *     that need device data (cu_seqlens, num_accepted) record a device error
 *     code that kda_read_device_error() / the decode error word returns.
 *   - Every device-side wait in the library is bounded; a wait that gives up
 *     records KDA_DEVERR_TIMEOUT instead of hanging.
 */
#ifndef KDA_H
#define KDA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same ABI as cudaStream_t. */
typedef struct CUstream_st *kda_stream_t;

enum kda_status {
    KDA_OK = 0,
    KDA_ERR_INVALID_ARG = 1,   /* null pointer, bad size, misaligned pointer   */
    KDA_ERR_UNSUPPORTED = 2,   /* D != 128, or a mode the library does not implement */
    KDA_ERR_CUDA = 3,          /* a CUDA runtime/driver call or launch failed   */
    KDA_ERR_TIMEOUT = 4,       /* a bounded device wait gave up                 */
    KDA_ERR_WORKSPACE = 5,     /* workspace missing or smaller than required    */
    KDA_ERR_DEVICE_CHECK = 6   /* device-side validation failed (see code)      */
};

enum kda_dtype { KDA_BF16 = 0, KDA_F32 = 1, KDA_E4M3 = 2 /* paged caches only */ };

/* Input options (bit flags), the kernel-side options of the pages' chunk_kda /
 * fused_recurrent_kda ("Kimi K3 模型结构（2）", section "训练、prefill、decode
 * 各用哪种形式": use_qk_l2norm_in_kernel, use_beta_sigmoid_in_kernel):
 *   KDA_FLAG_QK_L2NORM     q and k are divided by their L2 norm over the 128 key
 *                          channels, x / sqrt(sum(x^2) + 1e-6), per (token, head)
 *   KDA_FLAG_BETA_SIGMOID  beta holds logits; the kernels use 1 / (1 + exp(-beta))
 *   KDA_FLAG_CONV_SILU     kda_decode_step_fused only: SiLU, y / (1 + exp(-y)), after
 *                          the short convolution (the pages name no activation)
 *   KDA_FLAG_Q_SCALE       q is multiplied by d_k^-1/2 = 1 / sqrt(128) (after the L2
 *                          norm when both are set), the usual attention scale of the
 *                          chunk_kda interface; the pages give no scale, so it is off
 *                          by default (o = S^T q)
 * The decode cache keeps the projected inputs as given (unnormalised, logits). */
enum kda_flags {
    KDA_FLAG_QK_L2NORM = 1,
    KDA_FLAG_BETA_SIGMOID = 2,
    KDA_FLAG_CONV_SILU = 4,
    KDA_FLAG_Q_SCALE = 8
};

/* Device error codes (bit flags) written into the workspace / error word. */
enum kda_device_error {
    KDA_DEVERR_NONE = 0,
    KDA_DEVERR_CU_SEQLENS = 1,     /* cu_seqlens not 0 .. T_total, non-decreasing */
    KDA_DEVERR_NUM_ACCEPTED = 2,   /* num_accepted[b] outside 0 .. W-1            */
    KDA_DEVERR_TIMEOUT = 4,        /* a bounded wait gave up                       */
    KDA_DEVERR_LENGTHS = 8,        /* a length of the paged calls is negative, past the block table, or the
                                      new tokens do not add up to T_total           */
    KDA_DEVERR_NO_PAGES = 16,      /* the list of free pages is too short          */
    KDA_DEVERR_PAGE = 32,          /* a page or slot outside the cache             */
    KDA_DEVERR_TOKEN = 64,         /* a drafted token outside the vocabulary       */
    KDA_DEVERR_PROBS = 128         /* a row of probabilities without any weight    */
};

/* Human-readable name of a kda_status. Never NULL. */
const char *kda_status_string(int status);

/* Library ABI version (major * 100 + minor). */
int kda_version(void);

/* --------------------------------------------------------------------------
 * kda_chunk_fwd -- chunkwise prefill (chunk C = 64, 16-token sub-tiles).
 *
 * Defined by "Kimi K3 模型结构（2）", sections "UT 变换" and "块间递推与块内
 * 输出" (eqs. (4), (8)), computed in the matrix form of "Kimi K3: the Manos,
 * the Mythos ..." section "FlashKDA 算法":
 *   per chunk: U = (I+L)^{-1} Diag(beta) (V - K_decay S),
 *              O = Q_decay S + M_qk U,  S <- Diag(a_C) S + K_restore^T U,
 * with the 16-token sub-tile factorisation of "数值问题：1/Γ 会溢出" that the
 * bounded gate makes safe in bf16.  Packed documents restart the state at
 * every start given by cu_seqlens ("Kimi K3 模型结构（7）", section "文档边界").
 *
 *   q, k, v      (device) [T_total, H, D]  dtype
 *   z            (device) [T_total, H, D]  fp32 gate logits
 *   A            (device) [H]              fp32 per-head log scale A_h
 *   beta         (device) [T_total, H]     fp32, after sigmoid (logits with
 *                KDA_FLAG_BETA_SIGMOID)
 *   cu_seqlens   (device) int32 [n_seqs+1]: document offsets, cu[0] = 0,
 *                non-decreasing, cu[n_seqs] = T_total (empty documents allowed).
 *                NULL: n_seqs equal-length sequences (T_total % n_seqs == 0).
 *                Validated on the device: a bad array records
 *                KDA_DEVERR_CU_SEQLENS in the workspace and leaves o / final
 *                state unwritten.
 *   n_seqs       number of documents (>= 1)
 *   T_total      total tokens (>= 0, < 2^31)
 *   H            heads (>= 1);  D: must be 128
 *   dtype        KDA_BF16 or KDA_F32
 *   g_min        gate lower bound (the pages fix -5); must be in [-5, 0)
 *   flags        0 or an OR of KDA_FLAG_* (others: KDA_ERR_INVALID_ARG)
 *   init_state   (device) fp32 [n_seqs, H, D, D] or NULL (zeros)
 *   o            (device) [T_total, H, D] dtype, written
 *   final_state  (device) fp32 [n_seqs, H, D, D] or NULL (not written)
 *   workspace    (device) scratch of at least kda_chunk_fwd_workspace_size()
 *                bytes, 256-byte aligned; contents need no initialisation and
 *                are overwritten; must not be shared by calls in flight.
 * Pointers q, k, v, z, o must be 16-byte aligned.
 * ------------------------------------------------------------------------ */
size_t kda_chunk_fwd_workspace_size(int64_t T_total, int H, int n_seqs, int dtype);

/* --------------------------------------------------------------------------
 * kda_chunk_fwd_ckpt -- kda_chunk_fwd that also writes the state at
 * interval-aligned positions of every document ("Kimi K3 模型结构（7）",
 * section "混合架构的前缀缓存": a cached prefix is usable only where the KDA
 * state was persisted, so after each forward the kernel saves the state at
 * the last hash-aligned position, into a fresh slot).
 * Same arguments, checks and results as kda_chunk_fwd, plus
 *   ckpt_interval  tokens between checkpoints: a positive multiple of 64 (C)
 *   ckpt_slot      (device) int32 [n_seqs, ckpt_per_seq]: ckpt_slot[n][j] is
 *                  the page that receives the state of document n after its
 *                  first (j + 1) * ckpt_interval tokens; -1 (or any value
 *                  outside 0 .. n_slots - 1) skips it.  Positions past a
 *                  document's end are never written, so a caller that wants
 *                  only the last aligned state of each document marks only
 *                  that entry.
 *   ckpt_per_seq   columns of ckpt_slot (>= 1)
 *   ckpt           (device) fp32 [n_slots, H, D, D], 16-byte aligned: pages
 *   n_slots        pages in ckpt (>= 1)
 * Invalid checkpoint arguments return KDA_ERR_INVALID_ARG before any launch.
 * A call with checkpoints runs the same path as kda_chunk_fwd (fused launch,
 * three kernels or segments), in instantiations that carry the checkpoint
 * stores.
 * ------------------------------------------------------------------------ */
int kda_chunk_fwd_ckpt(const void *q, const void *k, const void *v,
                       const float *z, const float *A, const float *beta,
                       const int32_t *cu_seqlens, int n_seqs,
                       int64_t T_total, int H, int D, int dtype, float g_min,
                       const float *init_state, void *o, float *final_state,
                       int ckpt_interval, const int32_t *ckpt_slot, int ckpt_per_seq,
                       float *ckpt, int n_slots,
                       void *workspace, size_t workspace_bytes, int flags, kda_stream_t stream);

/* --------------------------------------------------------------------------
 * kda_chunk_fwd_plan_segments -- the segment count kda_chunk_fwd picks by
 * itself ("Kimi K3 模型结构（7）", section "KDA：三种执行形态" (SM-level CP):
 * when a few (document, head) chains over long documents would leave the
 * chain, not the parallel preparation, setting the time, kda_chunk_fwd runs
 * the kda_segment_scan decomposition with this many segments instead; its
 * results equal the single-chain run up to rounding).
 *   varlen  nonzero when the call passes cu_seqlens: the count for the
 *           longest document such a batch can hold (one of T_total tokens).
 *           The call itself plans from its actual longest document: when
 *           this bound is nonzero it reads cu_seqlens back to the host (it
 *           waits once for the stream; not while the stream is captured into
 *           a graph, which keeps the single-chain path).
 * Returns 0 for the single-chain path, else the segment count (2 .. 64).  The
 * choice depends on the shape, the dtype (bf16 only) and the current device's
 * SM count; kda_chunk_fwd_workspace_size already includes the room it needs
 * (a call given less keeps the single-chain path, with the same results).
 * No device work; never fails (invalid shapes return 0).
 * ------------------------------------------------------------------------ */
int kda_chunk_fwd_plan_segments(int64_t T_total, int H, int n_seqs, int dtype, int varlen);

/* The timing model behind that choice, measured on GB300: microseconds per
 * (chunk, head) preparation unit on one SM, and per chunk of one chain.  A
 * chain over L chunks is split when 1.3 us x L exceeds 1.5 times the
 * preparation time of the batch on the SMs the chains leave free.  NULL
 * arguments are skipped. */
void kda_planner_model(double *prep_us_per_unit, double *chain_us_per_chunk);

int kda_chunk_fwd(const void *q, const void *k, const void *v,
                  const float *z, const float *A, const float *beta,
                  const int32_t *cu_seqlens, int n_seqs,
                  int64_t T_total, int H, int D, int dtype, float g_min,
                  const float *init_state, void *o, float *final_state,
                  void *workspace, size_t workspace_bytes, int flags, kda_stream_t stream);

/* --------------------------------------------------------------------------
 * kda_chunk_fwd_noalloc -- kda_chunk_fwd without a caller-provided workspace.
 * The pages have no counterpart: this is an interface for callers that cannot
 * allocate device memory at call time (an engine that reserved the whole
 * device for its own pool, or a latency-critical path that cannot afford the
 * device synchronisation a cudaMalloc may imply).
 *
 * Same arguments, checks and results as kda_chunk_fwd, without workspace and
 * workspace_bytes.  It always runs the preparation and scan kernels one after
 * the other (never the single fused launch or the automatic segments), so its
 * results equal kda_chunk_fwd's up to rounding.  The workspace is a fixed array
 * of KDA_NOALLOC_SCRATCH_BYTES bytes in device global memory owned by the
 * library (every GPU that loads the library holds it until exit); the call
 * allocates nothing and calls no allocating routine.
 *   - The call needs the workspace of that sequential path: a header, the
 *     chunk table and one record per (chunk, head), with chunks =
 *     T_total / 64 + n_seqs (132,096 bytes per record in bf16, 164,352 in
 *     fp32).  A call needing more than KDA_NOALLOC_SCRATCH_BYTES returns
 *     KDA_ERR_WORKSPACE before any launch (about 500 (chunk, head) records in
 *     bf16, 400 in fp32).
 *   - The first call on a device looks up the array's device address (with
 *     that device current) and caches it with the device's CUDA context; a
 *     call under a new context (after a device reset) looks it up again.
 *     Make the first call on each device before any stream capture.
 *   - Every call uses the same array: calls whose executions overlap on the
 *     GPU race.  Order them, e.g. by issuing them on one stream.
 *   - Device-side errors (bad cu_seqlens, a timed-out wait) are recorded in
 *     the array's first word, which the next call clears;
 *     kda_noalloc_read_device_error() reads it.
 * ------------------------------------------------------------------------ */
#define KDA_NOALLOC_SCRATCH_BYTES (64ull << 20)

int kda_chunk_fwd_noalloc(const void *q, const void *k, const void *v,
                          const float *z, const float *A, const float *beta,
                          const int32_t *cu_seqlens, int n_seqs,
                          int64_t T_total, int H, int D, int dtype, float g_min,
                          const float *init_state, void *o, float *final_state,
                          int flags, kda_stream_t stream);

/* kda_noalloc_read_device_error -- synchronise `stream` and read the device
 * error code (bit flags of kda_device_error) that the last
 * kda_chunk_fwd_noalloc on the current device recorded in the library's
 * array.  Allocates nothing.  Returns KDA_OK, KDA_ERR_INVALID_ARG (code NULL)
 * or KDA_ERR_CUDA. */
int kda_noalloc_read_device_error(int32_t *code, kda_stream_t stream);

/* --------------------------------------------------------------------------
 * kda_segment_scan -- intra-device context parallelism over one long packed
 * token stream ("Kimi K3 模型结构（7）", section "KDA：三种执行形态" (SM-level
 * CP of long prefill), eq. (17) and "公式 (17) 的推导": segments are affine
 * maps S -> M S + S~; pairs compose as (M2,S~2) o (M1,S~1) = (M2 M1, M2 S~1 + S~2);
 * section "文档边界": only pairs of the same document are composed).
 *
 * The chunk list (documents cut into 64-token chunks, as in kda_chunk_fwd) is
 * split into n_segments contiguous, chunk-aligned ranges of balanced length
 * (earlier segments one chunk longer when the split is not exact).
 *   phase 1: every (head, segment) computes its pair (M, S~) from a zero state
 *            on its own SMs; a document start inside a segment resets the
 *            pair to (0, init_state[doc]) at that point;
 *   phase 2: entering states S_in[0] = 0, S_in[i+1] = M_i S_in[i] + S~_i;
 *   phase 3: every segment reruns from its exact entering state, writing o and
 *            the final state of every document that ends inside it.
 * Results equal kda_chunk_fwd on the same inputs up to rounding.
 *
 * Arguments as kda_chunk_fwd, plus
 *   n_segments   >= 1 (more segments than chunks leaves some empty), or 0 for
 *                the automatic count kda_segment_scan_auto_segments() returns
 *   pairs_M      (device) fp32 [H, n, D, D] or NULL: M of each segment
 *   pairs_S      (device) fp32 [H, n, D, D] or NULL: S~ of each segment
 *                (n = n_segments, or the automatic count)
 *   workspace    at least kda_segment_scan_workspace_size() bytes (same
 *                n_segments, 0 included).
 * ------------------------------------------------------------------------ */
size_t kda_segment_scan_workspace_size(int64_t T_total, int H, int n_seqs, int n_segments,
                                       int dtype);

/* The segment count kda_segment_scan takes for n_segments = 0: the most
 * segments whose rerun (two blocks per (segment, head)) fits in one wave of
 * the current device's SMs, at most sqrt(chunks / 6) (beyond it the
 * sequential composition costs more than the shorter chains save), at most 64
 * and half the chunks, at least 1; chunks = T_total / 64 + n_seqs.  No device
 * work; 0 for invalid shapes. */
int kda_segment_scan_auto_segments(int64_t T_total, int H, int n_seqs);

int kda_segment_scan(const void *q, const void *k, const void *v,
                     const float *z, const float *A, const float *beta,
                     const int32_t *cu_seqlens, int n_seqs,
                     int64_t T_total, int H, int D, int dtype, float g_min,
                     const float *init_state, int n_segments,
                     float *pairs_M, float *pairs_S,
                     void *o, float *final_state,
                     void *workspace, size_t workspace_bytes, int flags, kda_stream_t stream);

/* --------------------------------------------------------------------------
 * kda_decode_step -- one decode step with MTP draft replay ("Kimi K3 模型结构
 * （7）", section "KDA：三种执行形态，三种内核", decode paragraph: only the
 * projected inputs of draft tokens are cached; the accepted prefix is replayed
 * on chip, the bonus token is applied and the state is written back in place;
 * the next draft window runs speculatively in the same recurrence loop).
 * Per token the delta form of "Kimi K3: the Manos, the Mythos ..." section
 * "FlashKDA 算法": S <- D_t S; u = beta (v - S^T k); S <- S + k u^T; o = S^T q.
 *
 * A window holds W = 1 + n_draft tokens [t0, d1 .. d_{W-1}].  For each b:
 *   1. replay cache[b, 0 .. n_b - 1] (the drafts of the previous window that
 *      were accepted, n_b = num_accepted[b], 0 when num_accepted is NULL);
 *   2. apply t0 (bonus / next token), write o[b, 0], store the state in place;
 *   3. run d1 .. d_{W-1} from that state without storing it, write o[b, j];
 *   4. copy the projected inputs of d1 .. d_{W-1} into cache[b, 0 .. W-2].
 *
 *   state        (device) fp32 [N, H, D, D], read and written in place
 *   q, k, v      (device) [N, W, H, D] dtype;  z (device) fp32 [N, W, H, D]
 *   beta         (device) fp32 [N, W, H] (logits with KDA_FLAG_BETA_SIGMOID);
 *                A (device) fp32 [H]
 *   cache_q, cache_k, cache_v (device) [N, W-1, H, D] dtype, read and written
 *   cache_z      (device) fp32 [N, W-1, H, D]; cache_beta (device) fp32 [N, W-1, H]
 *                (the cache pointers may be NULL only when W == 1)
 *   num_accepted (device) int32 [N] with values in 0 .. W-1, or NULL
 *   N >= 1, H >= 1, D == 128, 1 <= W <= 8
 *   o            (device) [N, W, H, D] dtype, written
 *   error_word   (device) int32 or NULL: KDA_DEVERR_NUM_ACCEPTED is OR-ed in
 *                when a num_accepted value is out of range; that sequence's
 *                state, cache and outputs are then left untouched.
 *   flags        0 or an OR of KDA_FLAG_*, the same for every step of a
 *                sequence (the cache holds inputs as given)
 * state, q, k, v, z, o and the caches must be 16-byte aligned.
 * ------------------------------------------------------------------------ */
int kda_decode_step(float *state,
                    const void *q, const void *k, const void *v,
                    const float *z, const float *beta, const float *A,
                    void *cache_q, void *cache_k, void *cache_v,
                    float *cache_z, float *cache_beta,
                    const int32_t *num_accepted,
                    int N, int H, int D, int W, int dtype, float g_min,
                    void *o, int32_t *error_word, int flags, kda_stream_t stream);

/* --------------------------------------------------------------------------
 * kda_decode_step_fused -- the decode step with what the same paragraph puts
 * in the fused kernel around the recurrence ("Kimi K3 模型结构（7）", section
 * "KDA：三种执行形态，三种内核", decode: short convolution, input normalisation,
 * gate, KDA recurrence and output normalisation in one loop over the replayed
 * drafts, the bonus token and the next draft window).  The module around the
 * recurrence is the one of "Kimi K3: the Manos, the Mythos ..." section "Kimi
 * Linear": q, k, v pass a causal short convolution (left padding; width 4, as
 * in "Kimi K3 模型结构（7）", section "KDA 上下文并行", short-conv note) after
 * their projection; q and k are L2-normalised; the output is normalised per
 * head and scaled by an output gate.
 *
 * Per sequence b the committed stream continues the convolution state:
 * [conv_state (3 inputs), replayed drafts 0 .. n_b - 1, t0], and the window's
 * drafts follow t0.  Per token, in order:
 *   1. y_t = sum_{j<4} conv_w[., c, j] x_{t-3+j} per channel for each of q, k, v
 *      (pre-convolution inputs x come from the window or the cache), then SiLU
 *      with KDA_FLAG_CONV_SILU;
 *   2. the input options (KDA_FLAG_QK_L2NORM on the convolved q, k;
 *      KDA_FLAG_BETA_SIGMOID on beta);
 *   3. the recurrence exactly as kda_decode_step (replay, t0 committed in place,
 *      drafts speculative);
 *   4. o = o_raw / sqrt(mean_c(o_raw^2) + o_norm_eps) * o_norm_w[c] * sigmoid(o_gate)
 *      for the window's tokens, the mean over the 128 value channels of one
 *      (token, head).
 * The convolution state becomes the last three pre-convolution inputs of the
 * committed stream (ending at t0); the cache takes the window's drafts as given.
 *
 * Arguments as kda_decode_step, plus
 *   conv_w       (device) fp32 [3, H, D, 4]: taps of q, k, v per channel, tap 3
 *                on the current token (16-byte aligned)
 *   conv_state   (device) fp32 [N, H, 3, 3, D], read and written in place:
 *                q, k, v x the three latest committed inputs, oldest first
 *   o_gate       (device) fp32 [N, W, H, D]: output-gate logits
 *   o_norm_w     (device) fp32 [D]: output-norm weight (one vector for all heads)
 *   o_norm_eps   >= 0, added under the root
 *   flags        0 or an OR of KDA_FLAG_QK_L2NORM, KDA_FLAG_BETA_SIGMOID,
 *                KDA_FLAG_CONV_SILU
 * A sequence with an out-of-range num_accepted keeps its convolution state too.
 * ------------------------------------------------------------------------ */
int kda_decode_step_fused(float *state,
                          const void *q, const void *k, const void *v,
                          const float *z, const float *beta, const float *A,
                          const float *conv_w, float *conv_state,
                          const float *o_gate, const float *o_norm_w, float o_norm_eps,
                          void *cache_q, void *cache_k, void *cache_v,
                          float *cache_z, float *cache_beta,
                          const int32_t *num_accepted,
                          int N, int H, int D, int W, int dtype, float g_min,
                          void *o, int32_t *error_word, int flags, kda_stream_t stream);

/* ==========================================================================
 * The paged key/value cache of the full-attention layers that a hybrid model
 * puts between its linear-attention layers ("Kimi K3 模型结构（7）", section
 * "混合架构的前缀缓存": one page pool for the hybrid's layers, head-contiguous
 * pages).  Per serving step: kda_paged_tables once, then for every
 * full-attention layer kda_paged_append and kda_paged_attn.
 *
 * Conventions of the three calls
 *   - A cache (K or V) is [n_pages, Hkv, page_size, D]: one head's part of a
 *     page is contiguous.  Pages start page_stride elements apart
 *     (page_stride >= Hkv * page_size * D, a multiple of 16 bytes), so K and V
 *     may be two halves of one pool.  page_size is a multiple of 16, D is 128.
 *   - slot = page * page_size + offset (int64).
 *   - cache_dtype equals dtype, or is KDA_E4M3 with dtype KDA_BF16: the cache
 *     then holds x / scale rounded to e4m3 (saturating at +-448), with one
 *     fp32 scale per kv head for K and one for V.
 *   - Lengths, tables and slots live on the device and are checked there:
 *     what is wrong is OR-ed into error_word (device int32, or NULL), and is
 *     never used as an address.
 * ========================================================================== */

/* --------------------------------------------------------------------------
 * kda_paged_tables -- block tables, slot map, positions and offsets of a
 * step's new tokens, from the requests' lengths and a list of free pages.
 * Request i holds ctx_len[i] cached tokens and gains new_len[i]; with
 *   had = ceil(ctx / page_size), have = ceil((ctx + new) / page_size)
 * it takes have - had pages from the list, requests in order:
 *   block_table[i][b] = free_pages[f_i + b - had], had <= b < have,
 *   f_i = *free_head + sum_{j<i} (have_j - had_j).
 * Token t of request i (the new tokens packed in request order):
 *   positions[t] = ctx + t - cu_q[i],  slot_map[t] from block_table.
 *
 *   new_len, ctx_len (device) int32 [n_seqs], >= 0
 *   n_seqs       1 .. 16384;  T_total = sum of new_len, 0 <= T_total < 2^31
 *   block_table  (device) int32 [n_seqs, max_blocks]: entries 0 .. had - 1 are
 *                read where a token falls into a page that is not new, entries
 *                had .. have - 1 are written, the others are left alone
 *   free_pages   (device) int32 [n_free] (may be NULL when n_free is 0)
 *   free_head    (device) int32 [1]: entries of free_pages already taken
 *   free_head_next (device) int32 [1], written: free_head plus the pages taken
 *   slot_map     (device) int64 [T_total], written
 *   positions    (device) int32 [T_total] or NULL
 *   cu_q         (device) int32 [n_seqs + 1], written;  kv_len (device) int32
 *                [n_seqs], written: ctx + new
 * No output may be new_len, ctx_len, free_pages or free_head (blocks of one launch
 * read the one while another writes the other).
 * Lengths that are negative, exceed max_blocks * page_size or do not add up to
 * T_total record KDA_DEVERR_LENGTHS, too few free pages KDA_DEVERR_NO_PAGES.
 * Either makes the step an empty one: slot_map -1, positions 0, cu_q 0, kv_len =
 * ctx_len, free_head_next = *free_head, block_table as it was, so that
 * kda_paged_append writes nothing after it and kda_paged_attn has no rows.  A page
 * outside 0 .. n_pages - 1 records KDA_DEVERR_PAGE; its tokens get slot -1 and
 * a new entry becomes -1.
 * ------------------------------------------------------------------------ */
int kda_paged_tables(const int32_t *new_len, const int32_t *ctx_len, int n_seqs, int64_t T_total,
                     int32_t *block_table, int max_blocks, const int32_t *free_pages, int n_free,
                     const int32_t *free_head, int32_t *free_head_next, int page_size, int n_pages,
                     int64_t *slot_map, int32_t *positions, int32_t *cu_q, int32_t *kv_len,
                     int32_t *error_word, kda_stream_t stream);

/* --------------------------------------------------------------------------
 * kda_paged_append -- the new tokens' keys and values into the pages.
 *   k, v         (device) [T_total, Hkv, D] dtype, 16-byte aligned
 *   slot_map     (device) int64 [T_total]; a negative slot is skipped, one at or
 *                past n_pages * page_size is skipped and records KDA_DEVERR_PAGE;
 *                two tokens must not share a slot
 *   k_scale, v_scale (device) fp32 [Hkv], KDA_E4M3 only (else NULL), > 0 and finite
 *   k_cache, v_cache (device) the caches, written at the slots
 * ------------------------------------------------------------------------ */
int kda_paged_append(const void *k, const void *v, const int64_t *slot_map, int64_t T_total, int Hkv, int D,
                     int dtype, int cache_dtype, const float *k_scale, const float *v_scale, void *k_cache,
                     void *v_cache, int n_pages, int page_size, int64_t page_stride, int32_t *error_word,
                     kda_stream_t stream);

/* --------------------------------------------------------------------------
 * kda_paged_attn -- attention of every request's new tokens over its cached
 * keys (its new tokens' own keys among them: append first).
 * Request i's n_i = cu_q[i+1] - cu_q[i] queries stand at the positions
 * kv_len[i] - n_i .. kv_len[i] - 1; the query at position p sees the keys
 * max(0, p - window + 1) .. p (window 0: all up to p).  Query head h reads kv
 * head h / (Hq / Hkv).
 *   o   = softmax(sm_scale q K^T) V,   lse = log sum exp(sm_scale q K^T)
 * A query that sees no key (p < 0) gets o = 0, lse = -inf.
 *
 *   q            (device) [T_total, Hq, D] dtype, 16-byte aligned
 *   k_cache, v_cache, k_scale, v_scale, page_size, page_stride: as above; what
 *                the pages hold besides the keys that a new token of the request
 *                sees (NaN included) has no influence.  New tokens share products:
 *                a value that is not finite may make outputs of the request's other
 *                new tokens NaN too, where the mask hides it from them
 *   block_table  (device) int32 [n_seqs, max_blocks]; only the entries of pages
 *                that hold a seen key are read
 *   cu_q         (device) int32 [n_seqs + 1];  kv_len (device) int32 [n_seqs]
 *   max_q        the most new tokens of one request (0: not known, T_total)
 *   sm_scale     > 0 (1 / sqrt(128) is the usual one)
 *   o            (device) [T_total, Hq, D] dtype, written, 16-byte aligned
 *   lse          (device) fp32 [T_total, Hq] or NULL: natural logarithm
 *   workspace    kda_paged_attn_workspace_size() bytes, 256-byte aligned; needs
 *                no initialisation, not shared by calls in flight
 * A request whose offsets are not 0 <= cu_q[i] <= cu_q[i+1] <= T_total, or
 * that has over max_q tokens, records KDA_DEVERR_CU_SEQLENS and is left
 * out (its outputs are not written); a kv_len outside 0 .. max_blocks *
 * page_size records KDA_DEVERR_LENGTHS and counts as 0 (o = 0); a page outside
 * the cache records KDA_DEVERR_PAGE and that request's outputs are undefined.
 * The result does not depend on timing: the same call gives the same bits.
 * Roundings: o once, to dtype.  Over bf16 caches the probabilities are rounded to
 * bf16 before their product with V, over e4m3 caches to fp16 (2^-8 and 2^-11 of
 * each at most); the scores, their sums, the statistics, lse and o until its
 * rounding are fp32.  Over e4m3 caches q loses what is below 2^-31 of the largest
 * value of its row.  With dtype KDA_F32 everything is fp32.
 * ------------------------------------------------------------------------ */
size_t kda_paged_attn_workspace_size(int64_t T_total, int n_seqs, int Hq, int Hkv);

int kda_paged_attn(const void *q, const void *k_cache, const void *v_cache, const int32_t *block_table,
                   const int32_t *cu_q, const int32_t *kv_len, int n_seqs, int64_t T_total, int max_q, int Hq,
                   int Hkv, int D, int dtype, int cache_dtype, const float *k_scale, const float *v_scale,
                   int n_pages, int page_size, int64_t page_stride, int max_blocks, float sm_scale, int window,
                   void *o, float *lse, void *workspace, size_t workspace_bytes, int32_t *error_word,
                   kda_stream_t stream);

/* --------------------------------------------------------------------------
 * kda_paged_attn_sinks -- kda_paged_attn whose window leaves the first `sinks`
 * tokens of every request visible: the query at position p sees the keys
 *   0 .. min(sinks, p + 1) - 1  and  max(0, p - window + 1) .. p.
 * Everything else is as for kda_paged_attn (same workspace); sinks >= 0, and
 * sinks without a window change nothing.  A page that holds neither a sink nor
 * a key of some query's window is never read, and its table entry neither.
 * ------------------------------------------------------------------------ */
int kda_paged_attn_sinks(const void *q, const void *k_cache, const void *v_cache, const int32_t *block_table,
                         const int32_t *cu_q, const int32_t *kv_len, int n_seqs, int64_t T_total, int max_q, int Hq,
                         int Hkv, int D, int dtype, int cache_dtype, const float *k_scale, const float *v_scale,
                         int n_pages, int page_size, int64_t page_stride, int max_blocks, float sm_scale, int window,
                         int sinks, void *o, float *lse, void *workspace, size_t workspace_bytes,
                         int32_t *error_word, kda_stream_t stream);

/* ==========================================================================
 * Rotary positions and per-head norms of queries and keys, for the same
 * full-attention layers: kda_qk_rope alone, or kda_paged_rope_append, which also
 * does what kda_paged_append does.
 *
 * Per token t and head, over the 128 channels of a row x of q or k:
 *   1. with a weight w: x <- x / sqrt(mean(x^2) + eps) * w   (RMS norm)
 *   2. the first rot_dim channels are rot_dim / 2 pairs; pair i at position p
 *      is turned by the angle p f_i and multiplied by `amplitude`:
 *        (a, b) <- amplitude (a cos - b sin, a sin + b cos)
 *      KDA_ROPE_HALF: pair i is channels (i, i + rot_dim / 2);
 *      KDA_ROPE_INTERLEAVED: channels (2 i, 2 i + 1)
 * in fp32, rounded once at the end.  freq[i] is f_i in turns a position, times
 * 2^64 (kda_rope_frequencies): position times frequency is then exact modulo a
 * whole turn in 64-bit integers, at any position (negative ones too), and an
 * angle is off by less than 2^-25 radians from that however far the position.
 * Any table of frequencies will do, a model's own too.
 * ========================================================================== */
enum kda_rope_layout { KDA_ROPE_HALF = 0, KDA_ROPE_INTERLEAVED = 1 };
enum kda_rope_scaling { KDA_ROPE_NONE = 0, KDA_ROPE_LINEAR = 1, KDA_ROPE_NTK = 2, KDA_ROPE_YARN = 3 };

/* --------------------------------------------------------------------------
 * kda_rope_frequencies -- frequencies and amplitude, on the host, once per model.
 *   f_i = base^(-2 i / rot_dim), amplitude 1, for contexts stretched by `factor` (>= 1):
 *   KDA_ROPE_LINEAR  f_i / factor
 *   KDA_ROPE_NTK     base * factor^(rot_dim / (rot_dim - 2)) instead of base
 *   KDA_ROPE_YARN    f_i (g_i + (1 - g_i) / factor), where g_i goes linearly from 0 to 1
 *                    as the pair's turns over the original length, original_len f_i / 2 pi,
 *                    go from beta_slow to beta_fast; amplitude 0.1 ln(factor) + 1
 *                    (Peng et al., "YaRN: Efficient Context Window Extension of Large
 *                    Language Models", section 3).  This is the paper's text.  Many
 *                    checkpoints are trained with another ramp, linear in the pair's
 *                    number i between two whole pairs, and get frequencies from here that are
 *                    not theirs (base 10^6, factor 4, 32,768 positions, 128 channels: 16 of 64
 *                    pairs by over 1%, one by 42%): they take a table of their own, their f_i
 *                    / 2 pi times 2^64
 *   worked out in 64-bit floating point: within 2^-50 of f_i (2^-25 radians at p f_i = 2^25)
 *   rot_dim      a multiple of 8, 8 .. 128;  base > 1
 *   original_len, beta_fast, beta_slow   KDA_ROPE_YARN only: > 0, beta_fast > beta_slow >= 0
 *   freq         (host) int64 [rot_dim / 2], written;  amplitude (host), written
 * ------------------------------------------------------------------------ */
int kda_rope_frequencies(int rot_dim, double base, int scaling, double factor, double original_len, double beta_fast,
                         double beta_slow, int64_t *freq, float *amplitude);

/* --------------------------------------------------------------------------
 * kda_qk_rope
 *   q            (device) [T_total, Hq, D] dtype, tokens q_stride elements apart (>= Hq * D,
 *                a multiple of 16 bytes), so that q and k may be parts of one projection;
 *   k            (device) [T_total, Hkv, D], k_stride likewise
 *   positions    (device) int32 [T_total]
 *   freq         (device) int64 [rot_dim / 2]; rot_dim 0 (no rotation; freq and positions
 *                may be NULL) or a multiple of 8 up to 128
 *   amplitude    finite
 *   q_weight, k_weight  (device) fp32 [D] or NULL: no norm
 *   eps          >= 0
 *   q_out, k_out (device) as q and k, with strides of their own; may be q and k themselves
 *                (with their strides), and must not overlap the inputs otherwise
 * q, k, q_out, k_out, the weights and freq must be 16-byte aligned.
 * ------------------------------------------------------------------------ */
int kda_qk_rope(const void *q, const void *k, const int32_t *positions, const int64_t *freq, float amplitude,
                const float *q_weight, const float *k_weight, float eps, int64_t T_total, int Hq, int Hkv, int D,
                int rot_dim, int layout, int dtype, int64_t q_stride, int64_t k_stride, void *q_out, void *k_out,
                int64_t q_out_stride, int64_t k_out_stride, kda_stream_t stream);

/* --------------------------------------------------------------------------
 * kda_paged_rope_append -- kda_qk_rope with the keys written to their slots of the
 * paged cache instead of k_out, beside the values v (device) [T_total, Hkv, D] (v_stride
 * apart, as they are).  slot_map, caches, scales, page geometry and error_word as for
 * kda_paged_append; a skipped slot's query is still written to q_out.  An e4m3 cache
 * holds (the turned key) / scale, rounded once.
 * ------------------------------------------------------------------------ */
int kda_paged_rope_append(const void *q, const void *k, const void *v, const int32_t *positions,
                          const int64_t *slot_map, const int64_t *freq, float amplitude, const float *q_weight,
                          const float *k_weight, float eps, int64_t T_total, int Hq, int Hkv, int D, int rot_dim,
                          int layout, int dtype, int cache_dtype, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                          void *q_out, int64_t q_out_stride, const float *k_scale, const float *v_scale, void *k_cache,
                          void *v_cache, int n_pages, int page_size, int64_t page_stride, int32_t *error_word,
                          kda_stream_t stream);

/* --------------------------------------------------------------------------
 * kda_verify_drafts -- how many of each request's drafted tokens stand against the
 * target model's probabilities, and the token that follows them, by given uniform
 * numbers.  num_accepted is what the next kda_decode_step takes.
 * Request n with m drafts (d_0 .. d_{m-1}; p_j = target[n][j], the distribution after
 * d_0 .. d_{j-1}; q_j = draft[n][j], the distribution that d_j was drawn from):
 *   draft j stands when  u_j q_j(d_j) < p_j(d_j)  and all before it stand; a is their
 *   number.  The token after them is drawn by r = uniforms[n][W-1] from
 *     w = max(p_a - q_a, 0)   when draft a was refused (a < m; p_a where that is 0 all over),
 *     w = p_a                 when all stood (a = m):
 *   the lowest i with  sum_{k <= i} w_k > r sum_k w_k.
 * Without `draft` every draft is certain: q_j = 1 at d_j and 0 elsewhere.
 *   target       (device) [N, W, V] dtype, requests target_seq_stride and rows
 *                target_row_stride elements apart (>= V; padded vocabularies)
 *   draft        (device) [N, W-1, V] dtype, likewise, or NULL
 *   draft_tokens (device) int32 [N, W-1] (may be NULL when W is 1)
 *   uniforms     (device) fp32 [N, W], in [0, 1): u_0 .. u_{W-2}, r (r outside counts as 0
 *                below, as the largest number under 1 above)
 *   n_draft      (device) int32 [N], 0 .. W-1, or NULL: W-1 for all
 *   1 <= N <= 2^24, 1 <= W <= 32, 1 <= V < 2^31 - 4096; dtype KDA_F32 or KDA_BF16, values 0 .. 1
 *   num_accepted (device) int32 [N], written: a
 *   tokens       (device) int32 [N, W], written: d_0 .. d_{a-1}, the token drawn, then -1
 *   workspace    kda_verify_drafts_workspace_size() bytes, 8-byte aligned; needs no initialisation, not
 *                shared by calls in flight.  The size for N requests does for fewer (of this V and dtype) too
 * The tests are exact.  Weights are summed as multiples of 2^-60 (each, p - q exactly, rounded once),
 * so sums do not depend on their order and the same call gives the same tokens; as weights negative
 * values and NaN count as 0, and a test against NaN is refused.  A row with values of 2 and more, or one that sums to 8 or more, has no
 * answer (some token, or -1).
 * A drafted token outside 0 .. V-1 records KDA_DEVERR_TOKEN and is refused; its q_j counts as the row of
 * `draft` where there is one, and as 0 all over where drafts are certain.  An n_draft out
 * of range records KDA_DEVERR_NUM_ACCEPTED: that request gets num_accepted 0 and tokens -1.
 * Rows without weight record KDA_DEVERR_PROBS, and the token drawn is -1.
 * ------------------------------------------------------------------------ */
size_t kda_verify_drafts_workspace_size(int N, int W, int V, int dtype);

int kda_verify_drafts(const void *target, const void *draft, const int32_t *draft_tokens, const float *uniforms,
                      const int32_t *n_draft, int N, int W, int V, int dtype, int64_t target_seq_stride,
                      int64_t target_row_stride, int64_t draft_seq_stride, int64_t draft_row_stride,
                      int32_t *num_accepted, int32_t *tokens, void *workspace, size_t workspace_bytes,
                      int32_t *error_word, kda_stream_t stream);

/* --------------------------------------------------------------------------
 * kda_read_device_error -- synchronise `stream` and read the device error
 * code that the last kda_chunk_fwd / kda_segment_scan on `workspace`
 * recorded (bit flags of kda_device_error; 0 = none).
 * Returns KDA_OK, KDA_ERR_INVALID_ARG or KDA_ERR_CUDA.
 * ------------------------------------------------------------------------ */
int kda_read_device_error(const void *workspace, int32_t *code, kda_stream_t stream);

/* --------------------------------------------------------------------------
 * Diagnostics (no counterpart in the pages): per-launch timing and counting.
 *
 * kda_profile_enable(1) makes every following entry point record a CUDA event
 * on its stream before its first launch and after each of its kernel launches
 * (at most 256 marks are kept).  kda_profile_collect() synchronises on the
 * last mark, returns up to `max` (kernel name, milliseconds since the previous
 * mark) pairs in launch order, and clears the marks.  Names are static strings
 * owned by the library.  Returns the number of pairs, or -KDA_ERR_CUDA.
 * kda_launch_count() is the number of kernels the library has launched since
 * it was loaded (always counted, profiling or not).
 * ------------------------------------------------------------------------ */
int kda_profile_enable(int on);
int kda_profile_collect(const char **names, float *ms, int max);
long long kda_launch_count(void);

/* kda_set_wait_budget -- the clock-cycle limit of the library's waits on
 * flags that other blocks of the same launch raise (the fused prefill's
 * record-ready flags), of the decode's waits on its own copies and, where it is
 * under 10^6, of the paged attention's waits within its blocks, for every call
 * made afterwards in this process (not thread-safe against calls in
 * flight on other host threads).  A wait that runs out records
 * KDA_DEVERR_TIMEOUT (workspace error word, the call's error word), its block
 * stops, lets its own copies and tensor-core work finish and frees its TMEM,
 * and the call's outputs are then undefined.  cycles <= 0 restores the
 * default (2e9 cycles, about one second).  Returns the previous limit.  Meant
 * for tests of the timeout path; the other waits keep the default. */
long long kda_set_wait_budget(long long cycles);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H */
