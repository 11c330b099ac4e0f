/*
 * kda.h -- C ABI of the Kimi Delta Attention (KDA) library for one GB300 (sm_103a).
 *
 * KDA is a gated delta rule with channel-wise decay.  Per (sequence, head) it
 * carries a key-by-value state S (dk x dv, fp32) and, for each token t,
 *
 *     S_t = (I - beta_t k_t k_t^T) . Diag(exp g_t) . S_{t-1} + beta_t k_t v_t^T
 *     o_t = S_t^T q_t
 *
 * Sources (Kimi K3 report as summarised on the llm-atlas page "K3_RESEARCH.md"):
 * question ledger Q04 (fixed-shape recurrent state, channel-wise decay,
 * delta-rule write), Q05 (the write subtracts the state's prediction for the
 * current key), Q06 and Figure 3 (log-decay bounded below by g_min = -5 so the
 * diagonal tile can use BF16 tensor-core matmuls), Q07 (chunkwise-parallel
 * prefill with the state passed between chunks; O(1) state update for decode),
 * Q10 (attention output kept in FP32), and section 8's device layer ("fused
 * decode").  The agihunt digest page adds that FlashKDA cuts chunks further into
 * 16-token tiles for numerical stability.
 *
 * Conventions for every entry point:
 *   - All tensor pointers are caller-owned DEVICE memory of the current CUDA
 *     device, contiguous, 16-byte aligned (beta and cu_seqlens: 4-byte
 *     aligned) -- except for kda_prefill_host and kda_prefill_host_static, whose
 *     tensors are HOST memory.  The library allocates no memory per call: the
 *     host-buffer path creates its streams and events once per device, and
 *     kda_prefill_host_static's scratch is a fixed array in the library's image.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).
 *     Work is enqueued asynchronously on it; the call returns at once.
 *   - Argument errors are detected on the host and returned synchronously,
 *     before anything is enqueued.  A failed launch returns KDA_ERR_CUDA.
 *   - Errors found on the device (a bad cu_seqlens entry, a bounded wait that
 *     gave up) are recorded in a per-device status word; the affected work is
 *     skipped, nothing traps.  kda_last_device_status() reports and clears it.
 *   - q is not scaled (no 1/sqrt(dk)); callers pre-scale q if they want that.
 *   - Input prologue (the `prologue` word of kda_prefill_desc, kda_decode and
 *     kda_decode_multi; 0 = the inputs are used as given).  The workloads'
 *     input recipe -- q and k L2-normalised per (token, head), g = g_min *
 *     sigmoid(.), beta = sigmoid(.) -- can run inside the kernels' loads instead
 *     of as separate passes over HBM:
 *       KDA_PROLOGUE_QK_L2NORM   q and k are replaced by x / max(||x||_2, 1e-12)
 *                                over the dk channels of each (token, head),
 *                                computed in fp32 and rounded to qkv_dtype;
 *       KDA_PROLOGUE_G_LOGITS    g holds logits z; the decay used is -5 * sigmoid(z);
 *       KDA_PROLOGUE_BETA_LOGITS beta holds logits y; the write used is sigmoid(y).
 *   - Output gate (kda_prefill_gated, kda_decode_gated, kda_decode_multi_gated):
 *     the pages give KDA an input-dependent, full-rank gate over the read-out
 *     channels (llm-atlas Q08) but not its formula.  This library reads it as an
 *     elementwise sigmoid gate applied to the fp32 output, out = o * sigmoid(z),
 *     with the logits z [.., H, dv] fp32 computed by the caller (the projection
 *     that produces them is outside the attention kernel).  The gate changes only
 *     the written output, never the state.
 *   - Preconditions not checked on the host: g in [-5, 0] (the bounded
 *     log-decay; never clamped), beta in [0, 1].  Values outside these ranges
 *     are unsupported: they are computed, but without the accuracy bound.
 */
#ifndef KDA_H_
#define KDA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define KDA_ABI_VERSION 3

#define KDA_PROLOGUE_QK_L2NORM 1
#define KDA_PROLOGUE_G_LOGITS 2
#define KDA_PROLOGUE_BETA_LOGITS 4
#define KDA_PROLOGUE_ALL 7

typedef enum kda_status {
    KDA_OK = 0,
    KDA_ERR_INVALID_ARG = -1,   /* null/misaligned pointer, bad size, aliasing, bad cu_seqlens */
    KDA_ERR_UNSUPPORTED = -2,   /* head dims other than dk == dv in {64, 128}, unknown dtype */
    KDA_ERR_WORKSPACE = -3,     /* workspace smaller than kda_prefill_workspace_bytes() */
    KDA_ERR_CUDA = -4,          /* a CUDA runtime call or kernel launch failed */
    KDA_ERR_TIMEOUT = -5        /* a bounded on-device wait gave up (work skipped) */
} kda_status;

/* Storage type of q, k, v.  g, beta, states and outputs are always fp32. */
typedef enum kda_dtype {
    KDA_F32 = 0,
    KDA_BF16 = 1
} kda_dtype;

/* Shape of one prefill call. */
typedef struct kda_prefill_desc {
    int32_t num_seqs;       /* N >= 0 packed sequences */
    int32_t total_tokens;   /* T >= 0, sum of all sequence lengths */
    int32_t num_heads;      /* H >= 1 */
    int32_t dk;             /* key/query channels: 64 or 128 */
    int32_t dv;             /* value channels: must equal dk */
    int32_t qkv_dtype;      /* a kda_dtype */
    int32_t prologue;       /* KDA_PROLOGUE_* bits (0: inputs as given); others rejected */
} kda_prefill_desc;

/* Library ABI version (KDA_ABI_VERSION of the build). */
int32_t kda_abi_version(void);

/* Human-readable name of a status code (static string, never NULL). */
const char* kda_status_string(kda_status status);

/*
 * Bytes of device scratch memory kda_prefill needs for `desc` (may be 0).
 * Returns 0 for a desc that kda_prefill would reject.  Non-zero exactly when the
 * chunkwise form runs chunk-parallel: bf16, dk = dv = 128, at most 32768 (chunk, head)
 * items ((total_tokens / 64 + num_seqs) * num_heads), and a cost estimate from the shape
 * favours it over one CTA per (sequence, head): few units (up to ~130 for 8192-token
 * sequences), or a partial second wave on the 152 SMs.  The workspace then holds
 * the chunk offsets and, per (64-token chunk, head), the operands of that chunk's state
 * step: 115,200 bytes each, for (total_tokens / 64 + num_seqs) * num_heads chunks.
 */
size_t kda_prefill_workspace_bytes(const kda_prefill_desc* desc);

/* What one kda_prefill call for a given desc will do (for harnesses and tracing). */
typedef struct kda_prefill_plan {
    int32_t kernel_launches;   /* kernels one call enqueues */
    int32_t tensor_cores;      /* 1: BF16 tcgen05 path; 0: fp32 CUDA-core path */
    size_t workspace_bytes;    /* same as kda_prefill_workspace_bytes(desc) */
} kda_prefill_plan;

/*
 * Fills *plan for `desc`.  Host only, no CUDA call.  KDA_ERR_INVALID_ARG or
 * KDA_ERR_UNSUPPORTED for a desc that kda_prefill would reject.
 */
kda_status kda_prefill_query(const kda_prefill_desc* desc, kda_prefill_plan* plan);

/*
 * kda_prefill -- chunkwise-parallel KDA over varlen-packed sequences
 * (llm-atlas K3_RESEARCH.md, Q07: state passed recursively between chunks,
 * parallel matrix work inside a chunk; agihunt digest: 16-token tiles).
 *
 * Layouts (T = total_tokens, H = num_heads, N = num_seqs):
 *   q, k        [T, H, dk]   qkv_dtype
 *   v           [T, H, dv]   qkv_dtype
 *   g           [T, H, dk]   fp32, natural-log decay per key channel
 *   beta        [T, H]       fp32
 *   cu_seqlens  [N + 1]      int32, cu[0] = 0, non-decreasing, cu[N] = T;
 *                            NULL = N equal sequences (T % N must be 0)
 *   init_state  [N, H, dk, dv] fp32 (row c = key channel c); NULL = zero state
 *   out         [T, H, dv]   fp32, written for every token
 *   final_state [N, H, dk, dv] fp32; NULL = not written.  May be the same
 *                            pointer as init_state (in-place chaining of calls);
 *                            any other overlap with an input is rejected.
 *   workspace   device scratch of at least kda_prefill_workspace_bytes(desc)
 *               (may be NULL when that is 0), 16-byte aligned, overlapping no
 *               input or output; its contents need no set-up and are clobbered.
 *               Two calls in flight at once need two workspaces.  With a
 *               workspace the call computes chunk offsets, then the
 *               state-independent operands of every (chunk, head) at once and
 *               the state scan, in one cooperative launch at up to 120
 *               (sequence, head) units (two launches in all) or in two
 *               separate ones above that (three in all).  Without one, one
 *               launch.  All forms give bit-identical results.
 * A cu_seqlens entry that breaks the rules above is found on the device: that
 * sequence is skipped and kda_last_device_status() returns KDA_ERR_INVALID_ARG.
 */
kda_status kda_prefill(const kda_prefill_desc* desc,
                       const void* q, const void* k, const void* v,
                       const float* g, const float* beta,
                       const int32_t* cu_seqlens,
                       const float* init_state,
                       float* out, float* final_state,
                       void* workspace, size_t workspace_bytes,
                       void* stream);

/*
 * kda_prefill_gated -- kda_prefill with the output gate (see the top): every output
 * element is written as o * sigmoid(z), z = gate[t][h][j] (llm-atlas K3_RESEARCH.md, Q08,
 * read as an elementwise sigmoid gate on the read-out channels).
 *   gate  [T, H, dv] fp32 logits, device memory, 16-byte aligned; must not overlap out,
 *         final_state or the workspace.  NULL makes the call identical to kda_prefill.
 * Everything else (layouts, workspace, paths, errors) as kda_prefill; final_state is the
 * ungated recurrence's, bit for bit.
 */
kda_status kda_prefill_gated(const kda_prefill_desc* desc,
                             const void* q, const void* k, const void* v,
                             const float* g, const float* beta, const float* gate,
                             const int32_t* cu_seqlens,
                             const float* init_state,
                             float* out, float* final_state,
                             void* workspace, size_t workspace_bytes,
                             void* stream);

/*
 * kda_prefill_checkpointed -- kda_prefill that also snapshots each sequence's state at
 * chunk-aligned positions, for resuming a later request from a cached prefix (llm-atlas
 * K3_RESEARCH.md, Q31 hybrid prefix cache with sparse KDA checkpoints and 512-token hash
 * boundaries; section 8 device layer "KDA replay input"; Lab H boundary arithmetic).
 *
 * Same arguments and rules as kda_prefill, plus:
 *   checkpoint_interval  tokens between snapshots: a positive multiple of 64
 *   checkpoint_slots     snapshots kept per sequence (>= 1)
 *   checkpoints          [N, H, checkpoint_slots, dk, dv] fp32, device memory; slot j of
 *                        sequence n receives the state after its first (j + 1) *
 *                        checkpoint_interval tokens, for every such boundary that lies
 *                        within the sequence (the state after the whole sequence is
 *                        final_state).  Slots past a sequence's last boundary are not
 *                        written.  Must not overlap any other argument.
 * Resuming from slot j = running kda_prefill on the tokens after that boundary with
 * init_state = the snapshot.
 */
kda_status kda_prefill_checkpointed(const kda_prefill_desc* desc,
                                    const void* q, const void* k, const void* v,
                                    const float* g, const float* beta,
                                    const int32_t* cu_seqlens,
                                    const float* init_state,
                                    float* out, float* final_state,
                                    int32_t checkpoint_interval, int32_t checkpoint_slots,
                                    float* checkpoints,
                                    void* workspace, size_t workspace_bytes,
                                    void* stream);

/*
 * kda_prefill_host -- kda_prefill with q, k, v, g, beta, cu_seqlens, init_state, out and
 * final_state in HOST memory (same layouts and rules as kda_prefill; the chunkwise form
 * is the one of llm-atlas K3_RESEARCH.md, Q07).  The call walks the sequences in rounds of
 * `segment_tokens` tokens per sequence and keeps the state on the device between rounds:
 * round r's inputs are copied into one of two device staging sets on an upload stream
 * while round r-1 runs on `stream`, and round r-1's outputs are copied back on a
 * download stream (streams and events of the library, ordered after prior work on
 * `stream`).  segment_tokens is a positive multiple of 64, so the chunk boundaries, and
 * every output and final-state value, equal those of one kda_prefill call.
 *
 *   workspace   DEVICE memory of at least kda_prefill_host_workspace_bytes(desc,
 *               segment_tokens) bytes, 256-byte aligned; clobbered.
 *   stream      compute stream; when the call returns, `stream` has been made to wait for
 *               all of its copies and kernels: synchronise it before reading out or
 *               final_state, or reusing the host inputs.
 * Host buffers should be pinned (cudaHostAlloc / cudaHostRegister) for the copies to
 * overlap the kernels; pageable memory gives the same results more slowly.  Calls on one
 * device are serialised by the library while they enqueue.
 * Errors: as kda_prefill (cu_seqlens is checked on the host); KDA_ERR_INVALID_ARG for a
 * segment_tokens that is not a positive multiple of 64 or a misaligned workspace;
 * KDA_ERR_WORKSPACE for a short one.  Nothing is enqueued when an argument is rejected.  When
 * a CUDA call fails after work has been enqueued, the error is returned with `stream` made to
 * wait (as far as the runtime still allows) for the copies and kernels already enqueued, so
 * that synchronising it still marks the point after which no copy touches the buffers.
 */
size_t kda_prefill_host_workspace_bytes(const kda_prefill_desc* desc, int32_t segment_tokens);

kda_status kda_prefill_host(const kda_prefill_desc* desc,
                            const void* q, const void* k, const void* v,
                            const float* g, const float* beta,
                            const int32_t* cu_seqlens,
                            const float* init_state,
                            float* out, float* final_state,
                            int32_t segment_tokens,
                            void* workspace, size_t workspace_bytes,
                            void* stream);

/*
 * kda_prefill_host_static -- kda_prefill_host without a caller workspace.  The pages have
 * no counterpart to this entry point.  It is for callers that cannot call cudaMalloc when
 * a request arrives: a serving process that has already handed all of the device's memory
 * to its own pool (a fresh cudaMalloc would fail or fragment it), or a latency-bound loop
 * that cannot take the device-wide synchronisation a cudaMalloc may cause, and has no
 * device buffer of its own to lend.  The device staging then lives in a fixed scratch
 * array inside the library, KDA_STATIC_SCRATCH_BYTES per device, which every device that
 * loads the library holds until the process exits; the call itself calls no cudaMalloc,
 * cudaFree or allocating library routine.  Same arguments, layouts, results and stream
 * semantics as kda_prefill_host.
 *   - The first call on a device sets that device up (the scratch's device address, taken
 *     with cudaGetSymbolAddress while that device is current, and one event); make that
 *     first call before any stream capture.
 *   - Every call on a device shares the one array, which keeps whatever the last call left
 *     in it; each call writes every part of it that it reads (the state is copied in or
 *     zeroed first).  Two calls that ran on the GPU at the same time would race on it, so
 *     the library orders them: each call's copies and kernels run after those of the
 *     previous call on that device, whatever streams they were given.
 * Errors: as kda_prefill_host, and KDA_ERR_WORKSPACE when
 * kda_prefill_host_workspace_bytes(desc, segment_tokens) exceeds the scratch (a smaller
 * segment_tokens, or kda_prefill_host with a workspace, serves larger problems); nothing
 * is enqueued then.
 */
#define KDA_STATIC_SCRATCH_BYTES (64u << 20)

kda_status kda_prefill_host_static(const kda_prefill_desc* desc,
                                   const void* q, const void* k, const void* v,
                                   const float* g, const float* beta,
                                   const int32_t* cu_seqlens,
                                   const float* init_state,
                                   float* out, float* final_state,
                                   int32_t segment_tokens,
                                   void* stream);

/*
 * kda_decode -- one token per sequence, as a fused O(1) update of each head's
 * state: a single read and a single write of S (llm-atlas K3_RESEARCH.md, Q07
 * "decode keeps the O(1) state update"; section 8 device layer "fused decode").
 *
 * Layouts (B = batch):
 *   q, k   [B, H, dk]  qkv_dtype;     v [B, H, dv] qkv_dtype
 *   g      [B, H, dk]  fp32;          beta [B, H] fp32
 *   state  [B, H, dk, dv] fp32, read and overwritten in place
 *   out    [B, H, dv] fp32 (o = S_new^T q); must not overlap any input or state
 *   prologue  KDA_PROLOGUE_* bits applied to this token's inputs (see the top)
 */
kda_status kda_decode(int32_t batch, int32_t num_heads, int32_t dk, int32_t dv, int32_t qkv_dtype,
                      int32_t prologue,
                      const void* q, const void* k, const void* v,
                      const float* g, const float* beta,
                      float* state, float* out,
                      void* stream);

/*
 * kda_decode_gated -- kda_decode with the output gate: out = o * sigmoid(gate) elementwise
 * (llm-atlas K3_RESEARCH.md, Q08; see the top).  gate [B, H, dv] fp32 logits, device memory,
 * 16-byte aligned, overlapping neither out nor state; NULL = kda_decode.  The state update
 * is that of kda_decode, bit for bit.
 */
kda_status kda_decode_gated(int32_t batch, int32_t num_heads, int32_t dk, int32_t dv, int32_t qkv_dtype,
                            int32_t prologue,
                            const void* q, const void* k, const void* v,
                            const float* g, const float* beta, const float* gate,
                            float* state, float* out,
                            void* stream);

/*
 * kda_decode_multi -- K consecutive tokens of each sequence in one pass over each head's
 * state, for verifying K draft tokens (llm-atlas K3_RESEARCH.md, Q28: the MTP layer tuned
 * into an EAGLE-3 draft; Q07: O(1) decode update).  Per token the same fused update as
 * kda_decode; the state stays in registers across the K tokens, so HBM sees one read of
 * S and at most one write.
 *
 * Layouts (B = batch, K = tokens, 1 <= K <= KDA_DECODE_MULTI_MAX_TOKENS):
 *   q, k     [B, K, H, dk] qkv_dtype;   v [B, K, H, dv] qkv_dtype
 *   g        [B, K, H, dk] fp32;        beta [B, K, H] fp32
 *   n_apply  [B] int32 device memory, or NULL (= K for every sequence): the state of
 *            sequence b is replaced by the state after its first n_apply[b] tokens
 *            (0 leaves it untouched).  A value outside [0, K] leaves that state untouched
 *            and makes kda_last_device_status() return KDA_ERR_INVALID_ARG.
 *   state    [B, H, dk, dv] fp32, read, and written where n_apply[b] > 0
 *   out      [B, K, H, dv] fp32, o for every token (whatever n_apply says), or NULL
 * Verification: one call with n_apply = 0 (outputs for all K drafts, state untouched),
 * then one with n_apply = the accepted count per sequence and out = NULL.
 * prologue: KDA_PROLOGUE_* bits applied to every token's inputs (see the top).
 * Errors: as kda_decode, plus KDA_ERR_INVALID_ARG for K out of range.
 */
#define KDA_DECODE_MULTI_MAX_TOKENS 64

kda_status kda_decode_multi(int32_t batch, int32_t tokens, int32_t num_heads, int32_t dk, int32_t dv,
                            int32_t qkv_dtype, int32_t prologue,
                            const void* q, const void* k, const void* v,
                            const float* g, const float* beta,
                            const int32_t* n_apply,
                            float* state, float* out,
                            void* stream);

/*
 * kda_decode_multi_gated -- kda_decode_multi with the output gate on every token's output:
 * out = o * sigmoid(gate) (llm-atlas K3_RESEARCH.md, Q08; see the top).  gate [B, K, H, dv]
 * fp32 logits, device memory, 16-byte aligned, overlapping neither out nor state; ignored
 * when out is NULL; NULL = kda_decode_multi.  States as kda_decode_multi, bit for bit.
 */
kda_status kda_decode_multi_gated(int32_t batch, int32_t tokens, int32_t num_heads, int32_t dk, int32_t dv,
                                  int32_t qkv_dtype, int32_t prologue,
                                  const void* q, const void* k, const void* v,
                                  const float* g, const float* beta, const float* gate,
                                  const int32_t* n_apply,
                                  float* state, float* out,
                                  void* stream);

/*
 * kda_state_combine -- the fold step of context-parallel prefill over one long sequence
 * (llm-atlas K3_RESEARCH.md, section 8 system-state table: "KCP" in the pretraining row; Q07:
 * the state passed from chunk to chunk).  When consecutive token ranges of a sequence run on
 * different ranks, range r maps the state entering it as S_after = M_r S_before + S_r, where
 * M_r is the dk x dk product of its chunks' transitions (the state after the range from
 * initial state I with v = 0: kda_prefill with a zero v and an identity init_state) and S_r
 * is the state after the range from a zero start.  The state entering range r is then the
 * fold S <- M_j S + S_j over the ranges j < r, one call per step:
 *
 *   state_out[i] = transition[i] . state_in[i] + state_add[i]     for i < count (fp32)
 *
 *   count       number of (sequence, head) states, >= 0
 *   dk, dv      must be equal, 64 or 128 (else KDA_ERR_UNSUPPORTED)
 *   transition  [count, dk, dk] fp32, row-major (may be NULL when state_in is NULL)
 *   state_in    [count, dk, dv] fp32, row c = key channel c; NULL = zero
 *   state_add   [count, dk, dv] fp32; NULL = zero
 *   state_out   [count, dk, dv] fp32; may be state_add itself (in place), must not overlap
 *               state_in or transition (KDA_ERR_INVALID_ARG)
 * All pointers are device memory, 16-byte aligned; asynchronous on `stream`.
 */
kda_status kda_state_combine(int32_t count, int32_t dk, int32_t dv,
                             const float* transition, const float* state_in,
                             const float* state_add, float* state_out,
                             void* stream);

/*
 * ---- The draft step: operators around a tree of drafted tokens per sequence ----
 *
 * (llm-atlas K3_RESEARCH.md, Q28: draft tokens verified by the target; Q03 and Q31: KDA
 * layers beside attention layers with a paged cache.  Those layers are MLA there; the attention
 * here is that of key and value heads of one width, not of a latent cache.)  They share one description of the
 * trees, `parents` [B, K] int32, 1 <= K <= KDA_TREE_MAX_NODES:
 *   parents[b][i] = -1            node i follows the context
 *   0 <= parents[b][i] < i        node i follows that node
 *   parents[b][i] = KDA_TREE_PAD  there is no node i (trees of a batch may differ in size);
 *                                 no node may follow an absent one
 * A chain is parents[b][i] = i - 1.  A tree that breaks these rules is found on the device:
 * its sequence is skipped and kda_last_device_status() returns KDA_ERR_INVALID_ARG (what then
 * becomes of its outputs stands at each call).
 */
#define KDA_TREE_MAX_NODES 64
#define KDA_TREE_PAD (-2)

/*
 * kda_page_tables -- pages and slots for the tokens that a step appends to a paged cache,
 * built on the device from request lengths.  Request b has context_lens[b] tokens in the
 * cache, appends new_lens[b], and holds its first pages_held[b] table entries; the pages it
 * lacks are taken from free_pages in request order.
 *
 *   context_lens, new_lens, pages_held  [B] int32; pages_held covers the context
 *   block_table    [B, table_cols] int32, in place: the new pages' ids are written after the
 *                  held ones, nothing else is
 *   free_pages     [num_free] int32 page ids, taken from index 0 on (may be NULL when 0)
 *   slot_map       [max_tokens] int64: slot (page * page_size + offset) of every appended
 *                  token, request after request; -1 for a refused request's tokens and past the last
 *   cu_seqlens     [B + 1] int32: first appended token of each request (kda_prefill's layout)
 *   pages_held_out [B] int32;  pages_taken [1] int32: free_pages entries used up
 * A request whose tokens exceed its table row, or for which the free pages do not reach, is
 * refused: its pages_held_out is pages_held and its slots are -1.  Once the free pages have
 * not reached for one request, no later one takes any.  Negative lengths, or pages_held
 * that do not cover the context or exceed table_cols, make the request append nothing; more than max_tokens tokens leave
 * the rest without slots; both make kda_last_device_status() return KDA_ERR_INVALID_ARG.
 * No output may overlap an input or another output.  batch <= KDA_PAGE_TABLES_MAX_BATCH.
 */
#define KDA_PAGE_TABLES_MAX_BATCH 16384

kda_status kda_page_tables(int32_t batch, int32_t table_cols, int32_t num_free, int32_t page_size, int32_t max_tokens,
                           const int32_t* context_lens, const int32_t* new_lens, const int32_t* pages_held,
                           int32_t* block_table, const int32_t* free_pages,
                           int64_t* slot_map, int32_t* cu_seqlens, int32_t* pages_held_out, int32_t* pages_taken,
                           void* stream);

/* Shape of one kda_tree_attention call. */
typedef struct kda_tree_attention_desc {
    int32_t batch;          /* B >= 0 */
    int32_t nodes;          /* K, 1 .. KDA_TREE_MAX_NODES */
    int32_t num_heads;      /* query heads Hq, a multiple of num_kv_heads */
    int32_t num_kv_heads;   /* cache heads Hk >= 1 */
    int32_t dim;            /* channels per head: 64 or 128 */
    int32_t dtype;          /* a kda_dtype, of q, the caches and out */
    int32_t num_pages;      /* pages of the caches */
    int32_t page_size;      /* tokens of a page >= 1 */
    int32_t table_cols;     /* pages a sequence's table row can hold */
    float scale;            /* factor of the scores, finite */
    int64_t k_page_stride;  /* elements from one page to the next, >= page_size * Hk * dim, */
    int64_t v_page_stride;  /*   a multiple of 16 bytes */
} kda_tree_attention_desc;

/* Bytes of device scratch kda_tree_attention needs for `desc`; 0 for one it would reject. */
size_t kda_tree_attention_workspace_bytes(const kda_tree_attention_desc* desc);

/*
 * kda_tree_attention -- softmax attention of every node of every draft tree over a paged
 * key/value cache.  Node i of sequence b attends to the sequence's context_lens[b] cached
 * tokens and to the nodes on its own path from the context, itself included; node j's key
 * and value lie in the cache at logical position context_lens[b] + j.  K = 1 with parent -1
 * is single-token decode.
 *
 *   q             [B, K, Hq, dim] dtype
 *   k_cache, v_cache  page p, offset s, head h at p * page_stride + (s * Hk + h) * dim; query
 *                 head h reads cache head h / (Hq / Hk)
 *   block_table   [B, table_cols] int32: page of logical positions [j page_size, (j + 1) page_size)
 *   context_lens  [B] int32;  parents [B, K] int32
 *   out           [B, K, Hq, dim] dtype; zeros for absent nodes
 *   workspace     kda_tree_attention_workspace_bytes(desc) bytes, 16-byte aligned, clobbered;
 *                 two calls in flight at once need two
 * Whatever lies in the cache where a node may not look (past the last node, pages of others,
 * nodes of other paths) does not change its output, NaN included.  A sequence whose
 * context_lens is negative, or exceeds its table row or 2^31 - 8192 tokens with the K nodes added, or
 * whose tree is bad, gets zeros; a token whose page id is outside [0, num_pages) is left out; both make
 * kda_last_device_status() return KDA_ERR_INVALID_ARG.  Tables with room for more than 2^31
 * tiles of work (64 tokens of one block of rows; terabytes of cache) return
 * KDA_ERR_UNSUPPORTED.  bf16: the softmax's weights are
 * rounded to bf16 before they meet the values (their sum is kept in fp32), fp32: fp32 throughout.
 */
kda_status kda_tree_attention(const kda_tree_attention_desc* desc,
                              const void* q, const void* k_cache, const void* v_cache,
                              const int32_t* block_table, const int32_t* context_lens, const int32_t* parents,
                              void* out, void* workspace, size_t workspace_bytes, void* stream);

/*
 * kda_tree_decode -- KDA for every node of every draft tree from one read of the state: node
 * i's state is its parent's (the context's for parent -1) after one kda_decode step with its
 * own inputs.  The state is not changed; kda_tree_commit moves it.
 *
 *   q, k    [B, K, H, dk] qkv_dtype;  v [B, K, H, dv] qkv_dtype
 *   g       [B, K, H, dk] fp32;       beta [B, K, H] fp32
 *   parents [B, K] int32
 *   gate    [B, K, H, dv] fp32 logits of the output gate, or NULL
 *   state   [B, H, dk, dv] fp32, only read
 *   out     [B, K, H, dv] fp32, S_i^T q_i (gated);  zeros for absent nodes
 *   writes  [B, K, H, dv] fp32, beta_i (v_i - S'_i^T k_i) with S'_i the decayed state of
 *           the parent: what kda_tree_commit needs;  zeros for absent nodes
 * prologue as kda_decode.  out and writes overlap nothing.  Depth is not limited below K.
 * g may be -inf (or so low that e^g is zero): the node then starts from an empty state.  The rows of
 * out and writes of a sequence whose tree is bad are not written: they hold what they held.
 */
kda_status kda_tree_decode(int32_t batch, int32_t nodes, int32_t num_heads, int32_t dk, int32_t dv,
                           int32_t qkv_dtype, int32_t prologue,
                           const void* q, const void* k, const void* v, const float* g, const float* beta,
                           const int32_t* parents, const float* gate,
                           const float* state, float* out, float* writes, void* stream);

/*
 * kda_tree_commit -- each state moved to the end of an accepted path: after kda_tree_decode
 * on the same state with the same k, g and prologue, the state of node path[b][n_accept[b] - 1].
 *
 *   k [B, K, H, dk] qkv_dtype;  g [B, K, H, dk] fp32;  writes [B, K, H, dv] fp32
 *   path     [B, K] int32: the accepted nodes from the context on, in its first n_accept[b] entries
 *   n_accept [B] int32, 0 .. K; 0 leaves the state untouched
 *   state    [B, H, dk, dv] fp32 in place; overlaps nothing else
 * A path entry outside [0, K) or a count out of range leaves that state untouched and makes
 * kda_last_device_status() return KDA_ERR_INVALID_ARG.  prologue: the QK_L2NORM and G_LOGITS
 * bits (BETA_LOGITS is accepted and has no effect here).
 */
kda_status kda_tree_commit(int32_t batch, int32_t nodes, int32_t num_heads, int32_t dk, int32_t dv,
                           int32_t qkv_dtype, int32_t prologue,
                           const void* k, const float* g, const float* writes,
                           const int32_t* path, const int32_t* n_accept, float* state, void* stream);

/*
 * kda_verify_drafts -- which drafted tokens the target's probabilities keep, and the token
 * that follows them, from given random numbers.  From the context on, the children of the
 * current node are looked at in index order; child c with token x is kept when
 *     uniforms[c] * draft[c][x] < p[x]                             (draft given)
 *     uniforms[c] * m < p[x],  m = 1 - (p of the children before it)   (draft NULL)
 * with p the target's row of the current node; the walk goes on from a kept child.  Where
 * none is kept the next token is the argmax (lowest index first) of rest / noise: rest =
 * max(p - draft[c], 0) after a turned-down child c (draft given), p without the turned-down tokens
 * (draft NULL), p itself when there is none or nothing is left.  With noise ~ Exp(1) and
 * uniforms ~ U[0, 1) the kept tokens and the next one are distributed as the target's.
 * Every step is one IEEE fp32 operation per element.  A child whose token was turned down
 * at the same node before is passed over (draft NULL).
 *
 *   target   [B, K + 1, V] fp32: row 0 after the context, row i + 1 after node i; >= 0
 *   draft    [B, K, V] fp32: row i the distribution that node i's token was drawn from; then no
 *            two nodes may have the same parent.  NULL: tokens picked by rank or any other rule
 *   tokens, parents  [B, K] int32;  uniforms [B, K] fp32;  noise [B, V] fp32, > 0
 *   path     [B, K] int32: kept nodes in order, then -1;  n_accept [B] int32;  next_token [B] int32
 * path and n_accept are kda_tree_commit's; for chains n_accept is kda_decode_multi's n_apply.
 * A bad tree, or a token outside [0, V): path -1, n_accept 0, next_token -1, and
 * kda_last_device_status() returns KDA_ERR_INVALID_ARG.  V above KDA_VERIFY_MAX_VOCAB returns
 * KDA_ERR_UNSUPPORTED.
 */
#define KDA_VERIFY_MAX_VOCAB (1 << 30)

kda_status kda_verify_drafts(int32_t batch, int32_t nodes, int32_t vocab,
                             const float* target, const float* draft, const int32_t* tokens, const int32_t* parents,
                             const float* uniforms, const float* noise,
                             int32_t* path, int32_t* n_accept, int32_t* next_token, void* stream);

/*
 * ---- The attention layers' prompt path, and the upkeep of their cache ----
 *
 * (llm-atlas K3_RESEARCH.md, Q31 and section 8's serving engine: a paged cache whose prefixes are shared, copied on
 * write and given back; blog-mushroom and agihunt: long prompts taken in chunks.)  A prompt's chunk goes through an
 * attention layer as kda_page_tables (slots), kda_norm_rotate (queries ready, keys and values in the cache) and
 * kda_chunk_attention; single tokens and drafts as the same two and kda_tree_attention.
 */

/* Most query heads that may share a cache head in kda_chunk_attention. */
#define KDA_CHUNK_MAX_GROUP 64

/* Shape of one kda_chunk_attention call. */
typedef struct kda_chunk_attention_desc {
    int32_t batch;          /* B >= 0 */
    int32_t total_tokens;   /* T: rows of q and out */
    int32_t num_heads;      /* query heads Hq, a multiple of num_kv_heads */
    int32_t num_kv_heads;   /* cache heads Hk >= 1 */
    int32_t dim;            /* channels per head: 64 or 128 */
    int32_t dtype;          /* a kda_dtype, of q, the caches and out */
    int32_t num_pages;      /* pages of the caches */
    int32_t page_size;      /* tokens of a page >= 1 */
    int32_t table_cols;     /* pages a sequence's table row can hold */
    float scale;            /* factor of the scores, 2^126 in magnitude at most */
    int64_t k_page_stride;  /* elements from one page to the next, >= page_size * Hk * dim, */
    int64_t v_page_stride;  /*   a multiple of 16 bytes */
} kda_chunk_attention_desc;

/* Bytes of device scratch kda_chunk_attention needs for `desc`; 0 for one it would reject. */
size_t kda_chunk_attention_workspace_bytes(const kda_chunk_attention_desc* desc);

/*
 * kda_chunk_attention -- softmax attention of chunks of new tokens over a paged key/value cache.  Sequence b's
 * chunk is rows cu_seqlens[b] .. cu_seqlens[b + 1] of q; its token i stands at logical position context_lens[b] + i
 * and attends to the positions up to its own, whose keys and values (the chunk's own among them) are in the cache.
 * Chunks may differ in length; an empty one does nothing.
 *
 *   q             [T, Hq, dim] dtype
 *   k_cache, v_cache, block_table, context_lens   as kda_tree_attention's
 *   cu_seqlens    [B + 1] int32: 0 first, not decreasing, T at most (kda_page_tables' output)
 *   out           [T, Hq, dim] dtype; rows from cu_seqlens[B] on are left as they are
 *   workspace     kda_chunk_attention_workspace_bytes(desc) bytes (bf16, 128 channels: 40 to 324 MB, by the tokens and the cache),
 *                 16-byte aligned, clobbered; two calls in flight at once need two
 * Sequences of a few tokens each are served, but at 0.9 of kda_tree_attention's rate.
 * Whatever lies in the cache where a token may not look (behind it, pages of others) does not change its
 * output, NaN included.  A sequence whose context_lens is negative, or with its chunk exceeds its table row or
 * 2^31 - 8192 tokens, gets zeros; a token whose page id is outside [0, num_pages) is left out (a row that has nothing
 * else becomes zero); bad cu_seqlens leave out as it was; all make kda_last_device_status() return
 * KDA_ERR_INVALID_ARG.  A row whose visible scores are all -inf is NaN, as by the definition.
 * Weighted sums of values up to 2^82 (5e24) in magnitude stay finite whatever the scores and lengths; those of larger ones may
 * overflow where the definition does not.  bf16: the softmax's weights are rounded to bf16 before they meet the values (their sum is
 * kept in fp32), fp32: fp32 throughout.
 */
kda_status kda_chunk_attention(const kda_chunk_attention_desc* desc,
                               const void* q, const void* k_cache, const void* v_cache,
                               const int32_t* block_table, const int32_t* context_lens, const int32_t* cu_seqlens,
                               void* out, void* workspace, size_t workspace_bytes, void* stream);

/* Flags of kda_norm_rotate_desc. */
#define KDA_ROTATE_INTERLEAVED 1    /* pairs of channels (2i, 2i + 1) instead of (i, i + rot_dim / 2) */
#define KDA_ROTATE_NO_NORM 2        /* rotation only */

/* Shape of one kda_norm_rotate call. */
typedef struct kda_norm_rotate_desc {
    int32_t total_tokens;   /* T */
    int32_t num_heads;      /* query heads Hq */
    int32_t num_kv_heads;   /* cache heads Hk */
    int32_t dim;            /* channels per head: 64 or 128 */
    int32_t dtype;          /* a kda_dtype, of q, k, v, q_out and the caches */
    int32_t rot_dim;        /* channels that are rotated, the first ones: a multiple of 16, 0 .. dim */
    int32_t flags;          /* KDA_ROTATE_* */
    int32_t num_pages;      /* pages of the caches */
    int32_t page_size;      /* tokens of a page >= 1 */
    float eps;              /* of the norms, >= 0 */
    int64_t q_stride;       /* elements from one token to the next, >= its heads * dim, */
    int64_t k_stride;       /*   a multiple of 16 bytes: q, k and v may be parts of one */
    int64_t v_stride;       /*   projection's rows */
    int64_t k_page_stride;  /* as kda_tree_attention's */
    int64_t v_page_stride;
} kda_norm_rotate_desc;

/*
 * kda_norm_rotate -- queries and keys normed per head and rotated by their positions, keys and values written into the
 * cache, in one pass:
 *     y = x / sqrt(mean(x^2) + eps) * weight,   then for each pair (a, b) of rotated channels, with frequency f,
 *     (y_a, y_b) <- (y_a cos(p f) - y_b sin(p f), y_a sin(p f) + y_b cos(p f)),   p the token's position
 *
 *   q [T, Hq, dim], k, v [T, Hk, dim] dtype, tokens at their strides
 *   q_weight, k_weight  [dim] fp32, or NULL for ones
 *   inv_freq      [rot_dim / 2] fp32, radians a token (may be NULL when rot_dim is 0)
 *   positions     [T] int32 (may be NULL when rot_dim is 0)
 *   slots         [T] int64: where the token's key and value go (kda_page_tables' slot_map); negative:
 *                 nowhere.  No slot may come twice.
 *   q_out         [T, Hq, dim] dtype
 *   k_cache, v_cache  as kda_tree_attention's; only the slots' rows are written
 * fp32 arithmetic, rounded once; angles are exact to 1e-9 of a turn at any position, for frequencies up to 2^40 (a pair of an
 * infinite or NaN frequency is NaN).  A row's squares are summed in fp32: its elements stay below 1e18, and with eps 0 not all below 1e-18.
 * q_out overlaps nothing, the caches no input.  A slot past the caches is left out and makes
 * kda_last_device_status() return KDA_ERR_INVALID_ARG.
 */
kda_status kda_norm_rotate(const kda_norm_rotate_desc* desc, const void* q, const void* k, const void* v,
                           const float* q_weight, const float* k_weight, const float* inv_freq,
                           const int32_t* positions, const int64_t* slots,
                           void* q_out, void* k_cache, void* v_cache, void* stream);

/*
 * kda_page_fork -- table rows that share another row's first tokens.  Fork i gives the empty row children[i] the
 * first lens[i] tokens of row parents[i]: its whole pages by reference, and for a last page that they fill only partly a page of its
 * own, into which kda_cache_copy copies the rows.  lens[i] is at most what the parent has written: pages that it
 * holds past that (for drafts) cannot be told from others here, and a whole one would be shared although the parent appends
 * to it.  `shares` counts the rows that hold a page beyond the first, so that kda_page_release knows when it is free; pages of
 * kda_page_tables start at 0.
 *
 *   parents, children, lens  [num_forks] int32; a parent may come many times, a child once
 *   pages_held     [rows] int32; 0 for a child
 *   block_table    [rows, table_cols] int32, in place: the children's first entries are written
 *   shares         [num_pages] int32, in place
 *   free_pages     [num_free] int32 page ids, taken from index 0 on in the order of the forks (may be NULL when 0)
 *   pages_held_out [rows] int32: pages_held, and for the children what they hold now
 *   copies         [num_forks, 3] int32: source page, target page and rows to copy; (-1, -1, 0) for none
 *   pages_taken    [1] int32: free_pages entries used up
 * A fork for which the free pages do not reach is refused: its child stays empty, its copy is none; no later one takes a page
 * then.  A row out of range, a length that is negative or that the parent's pages do not cover, a child that
 * holds pages or comes twice, a parent that is a child in the same call: the fork does nothing.  A page id
 * out of range is passed on without a share.  Both make kda_last_device_status() return KDA_ERR_INVALID_ARG.
 * No output may overlap an input or another output.  num_forks <= rows <= KDA_PAGE_TABLES_MAX_BATCH.
 */
kda_status kda_page_fork(int32_t num_forks, int32_t rows, int32_t table_cols, int32_t num_pages, int32_t num_free, int32_t page_size,
                         const int32_t* parents, const int32_t* children, const int32_t* lens, const int32_t* pages_held,
                         int32_t* block_table, int32_t* shares, const int32_t* free_pages,
                         int32_t* pages_held_out, int32_t* copies, int32_t* pages_taken, void* stream);

/*
 * kda_page_release -- table rows cut to their first keep_lens tokens (0: given up; what the held pages hold, or more: untouched).
 * The pages behind those are given back: each loses a share, and those that no row holds any more are returned.
 *
 *   keep_lens, pages_held  [rows] int32
 *   block_table    [rows, table_cols] int32, only read: entries from pages_held_out on mean nothing afterwards
 *   shares         [num_pages] int32 >= 0, in place
 *   pages_held_out [rows] int32
 *   freed          [num_pages] int32: the freed pages in ascending order, then -1;  num_freed [1] int32
 * A row that would be cut inside a page which others hold as well is refused (what it appends there would be theirs:
 * kda_page_fork gives a row a copy); a negative length or pages_held out of range leave the row as it is; an
 * entry outside [0, num_pages) is passed over; a page given back more often than it is held is freed once.  All of
 * these make kda_last_device_status() return KDA_ERR_INVALID_ARG.  No output may overlap an input or another output.
 */
kda_status kda_page_release(int32_t rows, int32_t table_cols, int32_t num_pages, int32_t page_size,
                            const int32_t* keep_lens, const int32_t* pages_held, const int32_t* block_table,
                            int32_t* shares, int32_t* pages_held_out, int32_t* freed, int32_t* num_freed, void* stream);

/* The key/value caches of all layers that share their block tables.  Layer l, page p, offset s, head h begin at
 * l * layer_stride + p * page_stride + (s * num_kv_heads + h) * dim elements. */
typedef struct kda_cache_desc {
    int32_t num_layers;     /* >= 0 */
    int32_t num_pages;
    int32_t page_size;
    int32_t num_kv_heads;
    int32_t dim;            /* any, with rows of num_kv_heads * dim elements a multiple of 16 bytes */
    int32_t dtype;          /* a kda_dtype */
    int64_t k_layer_stride; /* of layers and of pages: elements, at least a page, a multiple of 16 bytes; */
    int64_t v_layer_stride; /*   not looked at where there is one layer, or one page */
    int64_t k_page_stride;
    int64_t v_page_stride;
} kda_cache_desc;

/*
 * kda_cache_copy -- rows of pages copied in every layer: the first copies[i][2] rows of page copies[i][0] to page
 * copies[i][1], keys and values.
 *
 *   copies  [num_copies, 3] int32, as kda_page_fork writes them; 0 rows: nothing
 *   k_cache, v_cache  in place
 * No target may come twice or be a source.  Pages out of range or more rows than a page has are
 * left out and make kda_last_device_status() return KDA_ERR_INVALID_ARG.
 */
kda_status kda_cache_copy(const kda_cache_desc* desc, int32_t num_copies, const int32_t* copies,
                          void* k_cache, void* v_cache, void* stream);

/*
 * kda_cache_keep_path -- the kept nodes' rows of a draft step moved to the front of the step's tokens, in every layer:
 * what kda_tree_commit does for the states.  For e < n_accept[b] the row of slots[b][path[b][e]] goes to
 * slots[b][e], as if all were read before any is written.
 *
 *   slots     [B, K] int64: where the step's nodes are in the cache; all different
 *   path      [B, K] int32, ascending in its first n_accept[b] entries;  n_accept [B] int32, 0 .. K
 *   k_cache, v_cache  in place
 * A path that does not ascend within [0, K), a count out of range, or a slot that is to move from or to somewhere outside the caches leaves
 * that sequence untouched and makes kda_last_device_status() return KDA_ERR_INVALID_ARG.
 */
kda_status kda_cache_keep_path(const kda_cache_desc* desc, int32_t batch, int32_t nodes, const int64_t* slots,
                               const int32_t* path, const int32_t* n_accept, void* k_cache, void* v_cache, void* stream);

/*
 * Synchronises `stream`, then returns and clears the device status word of the
 * current device: KDA_OK, KDA_ERR_INVALID_ARG (bad cu_seqlens seen on the
 * device) or KDA_ERR_TIMEOUT (a bounded wait gave up).  KDA_ERR_CUDA if the
 * synchronisation itself fails.
 */
kda_status kda_last_device_status(void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H_ */
