/*
 * kda.h — C ABI of the GB300 (sm_103a) Kimi Delta Attention forward library.
 *
 * The operation.  Each (sequence n, head h) unit keeps a d_k x d_v fp32 state S (rows are key
 * channels) and, token by token,
 *
 *     S_t = (I - beta_t k_t k_t^T) Diag(alpha_t) S_{t-1} + beta_t k_t v_t^T,   o_t = S_t^T q_t,
 *
 * with alpha_t = exp(log_alpha_t) one retention factor per key channel and beta_t a scalar
 * write strength.  Source: "How Kimi K3 Engineered Its Way to the Frontier"
 * (codepointer.substack.com), section "How KDA updates its state" (the report's formula and
 * the three-line token loop of flash-linear-attention's naive.py); restated in "Kimi K3"
 * (ai.thesatyajit.com), section "Kimi Delta Attention: constant-size memory over a million
 * tokens".  The interface mirrors FlashKDA's forward as described there (section "FlashKDA:
 * the equation, shipped as a kernel"): q, k, v, gate, beta, optional state in and out,
 * variable-length batching through cumulative sequence lengths, d = 128.
 *
 * Conventions shared by every entry point
 *   - Layouts are row-major and contiguous, batch folded into tokens:
 *       q, k, log_alpha : [T_tot, H, d_k]     v, out : [T_tot, H, d_v]     beta : [T_tot, H]
 *       states          : fp32 [N, H, d_k, d_v], row = key channel
 *   - Element type of q, k, v, log_alpha, beta and out: bf16 (KDA_BF16) or fp32 (KDA_FP32).
 *     log_alpha is the natural-log gate (alpha = exp(log_alpha), expected <= 0); beta is the
 *     write strength itself (already passed through a sigmoid).  No scale is applied to q.
 *   - Only d_k = d_v = 128 is supported.
 *   - Device tensors that a kernel reads or writes as 16-byte vectors must be 16-byte aligned
 *     (every torch allocation is); each entry point states which, and a misaligned one returns
 *     KDA_ERR_INVALID_ARG.  The prefill entry points need it for q, k, v, log_alpha, out and
 *     the states.
 *   - Ownership: the caller owns and allocates every buffer (device memory unless marked
 *     host).  The library never allocates or frees memory and keeps no per-call state; its
 *     only globals are the sticky device status word read by kda_read_device_status(), the
 *     fixed scratch array behind kda_fwd_chunked_noalloc() and the three streams per device
 *     of kda_fwd_chunked_host().
 *   - Every compute entry point but kda_fwd_chunked_host is asynchronous on `stream` (NULL =
 *     legacy default stream).  Host-side argument checks are synchronous and return before
 *     anything is launched.
 *   - With KDA_NVTX=1 in the environment (read once per process), every compute entry point
 *     wraps its launches in an NVTX range named after the entry point.
 *   - Errors: KDA_ERR_INVALID_ARG / KDA_ERR_UNSUPPORTED / KDA_ERR_WORKSPACE from the host
 *     checks, KDA_ERR_CUDA when a launch fails.  Conditions found on the device (a gate outside
 *     the supported domain, a bounded wait that gave up) set the sticky device status word;
 *     the kernels never trap or abort.
 */
#ifndef KDA_GB300_H
#define KDA_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t, declared without CUDA headers. */
typedef struct CUstream_st* kda_stream_t;

typedef enum kda_status {
    KDA_OK = 0,
    KDA_ERR_INVALID_ARG = -1,  /* null pointer, bad size, lengths not summing to T_tot     */
    KDA_ERR_UNSUPPORTED = -2,  /* d_k or d_v other than 128, unknown dtype                  */
    KDA_ERR_WORKSPACE = -3,    /* workspace missing or smaller than kda_fwd_workspace_bytes */
    KDA_ERR_CUDA = -4,         /* a CUDA launch or query failed                             */
    KDA_ERR_TIMEOUT = -5,      /* a bounded device-side wait gave up (device status word)   */
    KDA_ERR_DECAY_RANGE = -6   /* log_alpha > 0, or below -20 (see kda_fwd_chunked); in    */
                               /* kda_bwd, a 16-token chunk decaying beyond 160           */
} kda_status;

typedef enum kda_dtype { KDA_BF16 = 0, KDA_FP32 = 1 } kda_dtype;

/* Problem description.  host_seqlens is a HOST array of num_seqs lengths; it must equal the
 * differences of the device cu_seqlens array.  It lets the library size grids and workspace
 * without reading device memory.  The kernels check what they derive from the device array
 * against it before touching memory: a prefill CTA compares its sequence's length with the
 * host's (for calls of at most 2,048 sequences) and every derived offset (tokens, segment
 * workspace slots, checkpoint slots) with the host totals; the backward, decode-window and
 * fp32 prefill kernels check the token range and the workspace blocks.  A disagreement sets
 * KDA_ERR_INVALID_ARG in the device status word (read it with kda_read_device_status) and the
 * affected work item writes nothing. */
typedef struct kda_desc {
    int32_t num_seqs;            /* N >= 1                                            */
    int32_t num_heads;           /* H >= 1                                            */
    int64_t total_tokens;        /* T_tot = sum of host_seqlens                       */
    int32_t d_k;                 /* must be 128                                       */
    int32_t d_v;                 /* must be 128                                       */
    int32_t in_dtype;            /* kda_dtype of q, k, v, log_alpha, beta and out     */
    int32_t reserved;            /* must be 0                                         */
    const int32_t* host_seqlens; /* host, [num_seqs], each >= 0                       */
} kda_desc;

/* How a prefill call is split into work items (host-side plan, no device access). */
typedef struct kda_plan_info {
    int64_t chunks;           /* 64-token chunks summed over sequences (one head)          */
    int64_t work_items;       /* (sequence, segment) items per head                        */
    int32_t split_sequences;  /* sequences processed as more than one segment              */
    int32_t chunk_size;       /* tokens per chunk (64)                                     */
    int32_t segment_chunks;   /* longest segment of a split sequence, in chunks (0: none)  */
    int32_t reserved;
    size_t workspace_bytes;   /* what kda_fwd_chunked needs for this description           */
} kda_plan_info;

/*
 * kda_fwd_plan — fill *info with the work split of a prefill call.  Host only, no CUDA call.
 * Returns KDA_OK, KDA_ERR_INVALID_ARG or KDA_ERR_UNSUPPORTED.
 */
kda_status kda_fwd_plan(const kda_desc* desc, kda_plan_info* info);

/*
 * kda_fwd_workspace_bytes — bytes of device workspace kda_fwd_chunked needs for `desc`
 * (0 when no sequence is split into segments).  Host only.  Returns 0 for an invalid desc.
 */
size_t kda_fwd_workspace_bytes(const kda_desc* desc);

/*
 * kda_fwd_chunked — chunked prefill over packed variable-length sequences.
 *
 * Computes every o_t and, optionally, the final state of every (sequence, head) unit, exactly
 * as the token loop would, by the chunkwise form (64-token chunks aligned to each sequence's
 * own start; intra-chunk work as dense tensor-core tiles; one serial state step per chunk)
 * described in "How Kimi K3 Engineered Its Way to the Frontier", section "FlashKDA steps the
 * state once per 16 tokens".  Long sequences (above 65,536 tokens) are split into segments
 * whose transitions are evaluated independently of their incoming state and composed exactly
 * afterwards ("k3_training_and_infra_notes", section 4.1, intra-device context parallelism);
 * the segment count is a function of the sequence's length and the head count only (see
 * kda_fwd_plan), picked for the waves of GB300's 152 SMs.
 *
 *   desc          problem description (host)
 *   q, k, v, log_alpha, beta   device inputs, layouts above, element type desc->in_dtype
 *   init_state    device fp32 [N, H, 128, 128], or NULL for zeros.  May alias final_state.
 *   cu_seqlens    device int32 [N + 1], cu_seqlens[0] = 0, differences = host_seqlens
 *   out           device [T_tot, H, 128] of desc->in_dtype; must not alias any input
 *   final_state   device fp32 [N, H, 128, 128], or NULL to skip.  A zero-length sequence's
 *                 final state is its initial state.
 *   workspace     device scratch of at least kda_fwd_workspace_bytes(desc) bytes, 256-byte
 *                 aligned (NULL allowed when that size is 0).  Contents on entry are ignored.
 *   stream        CUDA stream the kernels are launched on.
 *
 * Bit-exactness: a sequence's results depend only on its own inputs and length, never on
 * the other sequences packed with it.
 *
 * Gate domain: every log_alpha in [-20, 0] is computed; this contains K3's bounded gate,
 * lower_bound * sigmoid(...) with lower_bound = -5 ("How Kimi K3 Engineered Its Way to the
 * Frontier", section "How KDA updates its state").  A chunk is a decay window: it starts where
 * the previous one ended, stays inside one 64-token block of the sequence, and is the longest
 * run of whole four-token groups (or the rest of the block) whose cumulative log-decay stays
 * within 80 in every channel, so every exponential factor of the chunkwise form is at most
 * e^40 in magnitude.  Ordinary gates give whole 64-token chunks; faster decay gives shorter
 * chunks (16 tokens at log_alpha = -5) and a proportionally slower call.  A positive log_alpha,
 * or a four-token group decaying by more than 80 in one channel (only possible below -20),
 * sets KDA_ERR_DECAY_RANGE in the device status word and leaves out and final_state
 * unspecified.  fp32 inputs (KDA_FP32) run the token loop itself in fp32, one pass over each
 * sequence, exact for every log_alpha <= 0 (no range applies).
 */
kda_status kda_fwd_chunked(const kda_desc* desc, const void* q, const void* k, const void* v,
                           const void* log_alpha, const void* beta, const float* init_state,
                           const int32_t* cu_seqlens, void* out, float* final_state,
                           void* workspace, size_t workspace_bytes, kda_stream_t stream);

/*
 * kda_fwd_checkpoint_count — number of states kda_fwd_chunked_ckpt writes for `desc` and an
 * interval of `ckpt_every` tokens: the sum over sequences of floor(L_n / ckpt_every).  Host
 * only.  Returns -1 if the description is invalid or ckpt_every is not a positive multiple of
 * 64 (the chunk size).
 */
int64_t kda_fwd_checkpoint_count(const kda_desc* desc, int32_t ckpt_every);

/*
 * kda_fwd_chunked_ckpt — kda_fwd_chunked that also writes state checkpoints.
 *
 * A prefix cache can resume a sequence only where its recurrent state was saved, and serving
 * saves it at the block-aligned positions a prefix lookup can reference
 * ("k3_training_and_infra_notes", section 4.5, KDA-aware prefix cache management; "How Kimi K3
 * Engineered Its Way to the Frontier", section "KDA states and MLA KV blocks share one paged
 * pool", Figure 12: a checkpoint at a 512-token hash-block boundary).  For every (sequence,
 * head) this call writes the fp32 state after the first p tokens, for p = ckpt_every,
 * 2 ckpt_every, ... up to and including the sequence length, in the layout of final_state.
 *
 *   ckpt_every    positive multiple of 64 (the chunk size), in tokens
 *   ckpt_states   device fp32 [count, H, 128, 128], count = kda_fwd_checkpoint_count(desc,
 *                 ckpt_every): sequence by sequence, each sequence's positions in increasing
 *                 order.  Must not alias any other argument; NULL only when count is 0.
 * Everything else (arguments, layouts, errors) is as for kda_fwd_chunked, and the outputs and
 * final states are bit-identical to that call's.  bf16 inputs only (KDA_ERR_UNSUPPORTED for
 * fp32 inputs).
 */
kda_status kda_fwd_chunked_ckpt(const kda_desc* desc, const void* q, const void* k,
                                const void* v, const void* log_alpha, const void* beta,
                                const float* init_state, const int32_t* cu_seqlens, void* out,
                                float* final_state, int32_t ckpt_every, float* ckpt_states,
                                void* workspace, size_t workspace_bytes, kda_stream_t stream);

/*
 * kda_fwd_chunked_noalloc — kda_fwd_chunked for callers that cannot allocate device memory.
 *
 * No counterpart in the paper: this is a deployment convenience.  Some callers cannot supply
 * the scratch workspace kda_fwd_chunked asks for, because they may not call cudaMalloc where
 * they run (inside an allocator or memory-pool callback, in a host that forbids device
 * allocation, or on a latency-critical path where an allocation could synchronise the
 * device).  This variant takes the same arguments minus the workspace and uses a scratch array
 * built into the library instead; it allocates nothing and calls no allocating routine.
 *
 *   - The scratch array is KDA_NOALLOC_SCRATCH_BYTES (48 MiB) of device memory that every GPU
 *     which loads this library holds until the process exits.
 *   - A call whose kda_fwd_workspace_bytes(desc) exceeds KDA_NOALLOC_SCRATCH_BYTES returns
 *     KDA_ERR_WORKSPACE before launching anything (the workspace holds 3 x 64 KiB per head
 *     and segment, so with H = 16 heads 16 segments fit in total).  Calls that need no
 *     workspace always run.
 *   - The first call on a device looks up the array's device address (cudaGetSymbolAddress,
 *     with that device current); make that first call before any stream capture.
 *   - Every call shares the one array and leaves its contents behind; nothing in it has to
 *     start at zero.  Calls that overlap on the GPU (different streams, or different host
 *     threads) race on the array: serialise them.
 * Everything else — arguments, layouts, results, errors — is as for kda_fwd_chunked.
 */
#define KDA_NOALLOC_SCRATCH_BYTES ((size_t)48 << 20)
kda_status kda_fwd_chunked_noalloc(const kda_desc* desc, const void* q, const void* k,
                                   const void* v, const void* log_alpha, const void* beta,
                                   const float* init_state, const int32_t* cu_seqlens, void* out,
                                   float* final_state, kda_stream_t stream);

/*
 * kda_fwd_host_workspace_bytes — bytes of device workspace kda_fwd_chunked_host needs for
 * `desc` cut into `parts` token-range parts.  Host only.  Returns 0 for an invalid desc or
 * part count.
 *
 * kda_fwd_chunked_host — kda_fwd_chunked on HOST buffers: uploads the inputs, runs the prefill
 * and downloads the results, overlapping the three.
 *
 * No counterpart in the paper: a caller whose tensors live in host memory would otherwise copy
 * everything up, compute, and copy everything down in turn.  The host link is the bound of such
 * a call, so the tokens are cut into parts and three streams of the library's own (created per
 * device on first use, kept for the process) overlap the upload of one part, the kernels of the
 * previous part and the download of the part before that.  Part j covers tokens [b_j, b_{j+1})
 * of every sequence longer than b_j; the boundaries are multiples of the 64-token chunk chosen
 * so that the parts hold about equal token counts, and no part spans more than 65,536 tokens
 * of a sequence (so more parts than asked for can run).  Each part's kernels are one
 * kda_fwd_chunked call whose initial states are the previous part's final states: a sequence
 * cut by a boundary is computed as a prefill resumed from its saved fp32 state, which agrees
 * with one kda_fwd_chunked call within rounding, not bit for bit.  A sequence that lies inside
 * the first part (for example every sequence, with parts = 1) gets the bits of kda_fwd_chunked.
 *
 *   desc          problem description (host), as for kda_fwd_chunked
 *   q, k, v, log_alpha, beta   HOST inputs, layouts and element type as for kda_fwd_chunked.
 *                 Page-locked (pinned) memory lets the copies run asynchronously and overlap;
 *                 pageable memory gives the same results with the copies serialised.
 *   init_state    HOST fp32 [N, H, 128, 128], or NULL for zeros
 *   out           HOST [T_tot, H, 128] of desc->in_dtype; must not overlap an input
 *   final_state   HOST fp32 [N, H, 128, 128], or NULL to skip
 *   parts         token-range parts, 1..64, or 0 for 8
 *   workspace     device scratch of at least kda_fwd_host_workspace_bytes(desc, parts) bytes,
 *                 256-byte aligned: the states in flight, every part's cumulative lengths and
 *                 three slots of one part's inputs and outputs.  Contents on entry are ignored.
 *   stream        the call's work starts after the work already queued on this stream.
 * Unlike the device entry points the call is synchronous: it returns when out and final_state
 * hold the results (or, after an error, when every copy it issued has finished).  Errors are
 * those of kda_fwd_chunked, plus KDA_ERR_WORKSPACE for a missing or small workspace and
 * KDA_ERR_CUDA for a failed copy or stream call.
 */
size_t kda_fwd_host_workspace_bytes(const kda_desc* desc, int32_t parts);
kda_status kda_fwd_chunked_host(const kda_desc* desc, const void* q, const void* k,
                                const void* v, const void* log_alpha, const void* beta,
                                const float* init_state, void* out, float* final_state,
                                int32_t parts, void* workspace, size_t workspace_bytes,
                                kda_stream_t stream);

/*
 * kda_decode_step — one decode token per (sequence, head), state updated in place.
 *
 * For every unit: S <- Diag(exp(g)) S;  u = beta (v - S^T k);  S <- S + k u^T;  o = S^T q.
 * The state is read once and written once ("k3_training_and_infra_notes", section 4.5, KDA
 * decoding: the recurrent state is updated in place at every decoding step).
 *
 *   desc          num_seqs = N, total_tokens = N; host_seqlens may be NULL (all lengths 1)
 *   q, k, log_alpha  device [N, H, 128];  v: [N, H, 128];  beta: [N, H]  (desc->in_dtype)
 *   state         device fp32 [N, H, 128, 128], read and overwritten in place
 *   out           device [N, H, 128] of desc->in_dtype; must not alias any input
 */
kda_status kda_decode_step(const kda_desc* desc, const void* q, const void* k, const void* v,
                           const void* log_alpha, const void* beta, float* state, void* out,
                           kda_stream_t stream);

/*
 * kda_decode_window — a run of decode tokens per sequence in one pass over the state.
 *
 * Speculative decoding verifies a window of drafted tokens and must then move each state to
 * the last accepted token.  The state after any accepted prefix follows from the drafted
 * tokens' projected inputs, which are far smaller than the state, so only those are cached:
 * the accepted tokens are replayed on-chip together with the bonus token and the next draft
 * window in one recurrent loop, and the state is written back once
 * ("k3_training_and_infra_notes", section 4.5, KDA decoding).  For every (sequence, head):
 * starting from `state`, the tokens of sequence n (rows cu_seqlens[n] .. cu_seqlens[n+1] - 1)
 * run through the recurrence of kda_decode_step one after another; each token's output is
 * computed from the state after the tokens before it; the state after the first commit[n]
 * tokens is written back.
 *
 *   desc          num_seqs = N; host_seqlens required: per-sequence run lengths, 0 .. 64
 *   q, k, log_alpha, v  device [T, H, 128];  beta: [T, H]  (T = total_tokens, desc->in_dtype)
 *   cu_seqlens    device int32 [N + 1], differences = host_seqlens
 *   state         device fp32 [N, H, 128, 128]; overwritten with the state after the first
 *                 commit[n] tokens of run n, left untouched when that count is 0
 *   out           device [T, H, 128] of desc->in_dtype, or NULL to skip the outputs
 *   commit        device int32 [N] (each clamped to 0 .. run length), or NULL to commit every
 *                 token
 * A run of one token with commit 1 gives the bits of kda_decode_step.
 */
kda_status kda_decode_window(const kda_desc* desc, const void* q, const void* k, const void* v,
                             const void* log_alpha, const void* beta, const int32_t* cu_seqlens,
                             float* state, void* out, const int32_t* commit, kda_stream_t stream);

/*
 * Input prologue: the recurrence's inputs from a layer's raw per-token projections.
 *
 * Queries and keys of a KDA layer pass through Swish and are then L2-normalised over their
 * 128 channels; values pass through Swish ("Kimi K3" (ai.thesatyajit.com), section "Kimi Delta
 * Attention: constant-size memory over a million tokens").  The decay is K3's gate with a lower
 * bound, log_alpha = lower_bound * sigmoid(exp(A_log[h]) * (g_raw + dt_bias[h, :])), which keeps
 * every log_alpha inside (lower_bound, 0) ("How Kimi K3 Engineered Its Way to the Frontier",
 * section "How KDA updates its state").  beta arrives as logits and passes through a sigmoid
 * (FlashKDA's forward, section "FlashKDA: the equation, shipped as a kernel").  Readings where
 * the sources are silent: the L2 norm divides by sqrt(sum of squares + 1e-6); q is multiplied
 * by q_scale after its norm.  The short convolution that precedes Swish in the layer is the
 * caller's: the raw q, k, v here are its outputs.
 *
 * Arithmetic (fp32, every result rounded to bf16 where an unfused pipeline would store it):
 *   sigmoid(x) = 1 / (1 + 2^(-x log2 e)) with the hardware exp2 and reciprocal approximations
 *   (about 1e-6 relative error); Swish(x) = x sigmoid(x); the row norm sums the squares of eight
 *   consecutive channels in order and then adds the sixteen partial sums pairwise (strides 1,
 *   2, 4, 8).
 */
typedef struct {
  const float* A_log;    /* device fp32 [H]: per-head log decay rate */
  const float* dt_bias;  /* device fp32 [H, 128], or NULL for none */
  float lower_bound;     /* in [-80, 0): most negative log_alpha (K3 uses -5); the chunked
                            prefill computes log_alpha >= -20 (see kda_fwd_chunked) */
  float q_scale;         /* finite, > 0: factor on the normalised q (1/sqrt(128) is usual) */
} kda_prologue_params;

/*
 * kda_prologue — the prologue alone, as an elementwise pass over HBM (for decode steps and
 * windows, or any caller that wants the transformed inputs).
 *
 *   desc          total_tokens rows, num_heads heads; in_dtype must be KDA_BF16;
 *                 host_seqlens unused (may be NULL)
 *   q_raw, k_raw, v_raw, g_raw   device bf16 [T, H, 128]
 *   beta_logit    device bf16 [T, H]
 *   q, k, v, log_alpha           device bf16 [T, H, 128] outputs
 *   beta          device bf16 [T, H] output
 * Outputs must not alias inputs or each other.  Returns KDA_ERR_UNSUPPORTED for fp32 inputs.
 */
kda_status kda_prologue(const kda_desc* desc, const kda_prologue_params* prm, const void* q_raw,
                        const void* k_raw, const void* v_raw, const void* g_raw,
                        const void* beta_logit, void* q, void* k, void* v, void* log_alpha,
                        void* beta, kda_stream_t stream);

/*
 * kda_prologue_conv — the short convolution of q, k and v, then the prologue, as one pass.
 *
 * A KDA layer produces q, k and v by a short convolution followed by the prologue ("Kimi K3"
 * (ai.thesatyajit.com), section "Kimi Delta Attention…"); the convolution is causal and
 * depthwise with kernel size 4, and serving keeps three of its caches per request and layer
 * ("How Kimi K3 Engineered Its Way to the Frontier", section "What the hybrid saves": 216 KiB per
 * layer in bf16).  Per (sequence, head, channel): y_t = sum_{j=0..3} w[j] x_{t-3+j}, no bias,
 * w[3] on the current token, inputs before the sequence's first token from the cache (zeros when
 * cache_in is NULL); accumulated in fp32 in the order j = 0..3 and passed to the prologue
 * unrounded.  log_alpha and beta get no convolution.
 *
 *   desc          as for kda_fwd_chunked (host_seqlens required); in_dtype KDA_BF16
 *   conv->w_q, w_k, w_v   device fp32 [H, 128, 4], 16-byte aligned
 *   conv->cache_in        device bf16 [N, 3, 3, H, 128] (tensor q/k/v, then the 3 inputs before
 *                         each sequence, oldest first), or NULL for zeros
 *   conv->cache_out       device bf16, same layout: each sequence's last 3 raw inputs after the
 *                         call (continuing from cache_in when shorter), or NULL; may equal
 *                         cache_in (updated in place)
 *   cu_seqlens    device int32 [N+1]
 * Other arguments and outputs as for kda_prologue.  The outputs feed kda_fwd_chunked (or the
 * decode calls); a run split into consecutive calls with the cache carried equals one call.
 */
typedef struct {
  const float* w_q;      /* device fp32 [H, 128, 4] */
  const float* w_k;
  const float* w_v;
  const void* cache_in;  /* device bf16 [N, 3, 3, H, 128] or NULL */
  void* cache_out;       /* device bf16 [N, 3, 3, H, 128] or NULL; may equal cache_in */
} kda_conv_params;

kda_status kda_prologue_conv(const kda_desc* desc, const kda_prologue_params* prm,
                             const kda_conv_params* conv, const int32_t* cu_seqlens,
                             const void* q_raw, const void* k_raw, const void* v_raw,
                             const void* g_raw, const void* beta_logit, void* q, void* k, void* v,
                             void* log_alpha, void* beta, kda_stream_t stream);

/*
 * kda_fwd_chunked_prologue — kda_fwd_chunked on raw projections, with the prologue fused into
 * the prefill's load path: the transformed q, k, v, log_alpha and beta never go to HBM.
 *
 * Arguments as kda_fwd_chunked, with q_raw, k_raw, v_raw, g_raw and beta_logit (layouts as q, k,
 * v, log_alpha and beta) in place of the transformed inputs and `prm` as for kda_prologue.
 * Outputs and final states are bit-identical to kda_prologue followed by kda_fwd_chunked.
 * bf16 inputs only (KDA_ERR_UNSUPPORTED for fp32 inputs).
 */
kda_status kda_fwd_chunked_prologue(const kda_desc* desc, const kda_prologue_params* prm,
                                    const void* q_raw, const void* k_raw, const void* v_raw,
                                    const void* g_raw, const void* beta_logit,
                                    const float* init_state, const int32_t* cu_seqlens, void* out,
                                    float* final_state, void* workspace, size_t workspace_bytes,
                                    kda_stream_t stream);

/*
 * kda_decode_step_prologue, kda_decode_window_prologue — kda_decode_step and kda_decode_window
 * on raw projections, with the input prologue (as for kda_prologue) fused into the decode kernels:
 * K3's decode reads a token's projected inputs and normalises and gates them on-chip in the same
 * kernel as the recurrence ("k3_training_and_infra_notes", section 4.5, KDA decoding).
 *
 * Arguments as kda_decode_step / kda_decode_window, with q_raw, k_raw, v_raw, g_raw and
 * beta_logit in place of q, k, v, log_alpha and beta, and `prm` as for kda_prologue; q_raw and
 * k_raw must be 16-byte aligned (KDA_ERR_INVALID_ARG otherwise).  Outputs and states are
 * bit-identical to kda_prologue followed by the plain call.  bf16 inputs only
 * (KDA_ERR_UNSUPPORTED for fp32 inputs).
 */
kda_status kda_decode_step_prologue(const kda_desc* desc, const kda_prologue_params* prm,
                                    const void* q_raw, const void* k_raw, const void* v_raw,
                                    const void* g_raw, const void* beta_logit, float* state,
                                    void* out, kda_stream_t stream);
kda_status kda_decode_window_prologue(const kda_desc* desc, const kda_prologue_params* prm,
                                      const void* q_raw, const void* k_raw, const void* v_raw,
                                      const void* g_raw, const void* beta_logit,
                                      const int32_t* cu_seqlens, float* state, void* out,
                                      const int32_t* commit, kda_stream_t stream);

/*
 * kda_bwd — gradients of the recurrence (the backward pass) for training.
 *
 * For the forward of kda_fwd_chunked (the token loop of "How Kimi K3 Engineered Its Way to the
 * Frontier", section "How KDA updates its state") and the gradient d_out of a loss with respect to
 * every output (and optionally d_state with respect to the final states), returns the gradients
 * with respect to q, k, v, log_alpha, beta and the initial states.  Chunked by 16 tokens (the
 * pages' state step, "FlashKDA steps the state once per 16 tokens"), on tensor cores (tf32
 * operands, fp32 accumulation): a forward pass stores the state at every chunk start, a reverse
 * pass carries the gradient of the state backwards and computes each chunk's gradients.
 * Domain: in every 16-token chunk, every key channel decays by at most 160 (a mean log_alpha of
 * -10 per token, twice the bounded gate's floor of -5); a chunk beyond that sets
 * KDA_ERR_DECAY_RANGE in the device status word and its gradients are then unspecified.
 *
 *   desc          as for kda_fwd_chunked (host_seqlens required); q, k, v, log_alpha, beta of
 *                 desc->in_dtype, layouts as there; q, k, v, log_alpha 16-byte aligned
 *   init_state    device fp32 [N, H, 128, 128] or NULL (zeros)
 *   d_out         device fp32 [T, H, 128]
 *   d_state       device fp32 [N, H, 128, 128] or NULL (no loss on the final states)
 *   dq, dk, dv, dlog_alpha   device fp32 [T, H, 128]; dbeta device fp32 [T, H];
 *   dinit_state   device fp32 [N, H, 128, 128]
 *   workspace     device, at least kda_bwd_workspace_bytes(desc) bytes, 16-byte aligned: the
 *                 sequences' chunk offsets, then per 16-token chunk and head three 16 x 16 fp32
 *                 tiles, the chunk's start state (128 x 128 fp32) and a 16 x 128 fp32 tile;
 *                 contents on return are unspecified
 * The gradients are deterministic (no atomics; every sum runs in a fixed order).  If the device
 * cu_seqlens disagree with the host lengths in their chunk total or run past T, the first launch
 * sets KDA_ERR_INVALID_ARG in the device status word, nothing else is computed and every output
 * is unspecified.  Outputs must not alias inputs or each other.  Argument, alignment and
 * workspace errors return KDA_ERR_INVALID_ARG / KDA_ERR_WORKSPACE before anything is launched.
 */
size_t kda_bwd_workspace_bytes(const kda_desc* desc);
kda_status kda_bwd(const kda_desc* desc, const void* q, const void* k, const void* v,
                   const void* log_alpha, const void* beta, const float* init_state,
                   const int32_t* cu_seqlens, const float* d_out, const float* d_state, float* dq,
                   float* dk, float* dv, float* dlog_alpha, float* dbeta, float* dinit_state,
                   void* workspace, size_t workspace_bytes, kda_stream_t stream);

/*
 * Paged serving of the layers next to KDA.
 *
 * A hybrid model keeps KDA states and the keys and values of its full-attention layers in one
 * paged pool ("How Kimi K3 Engineered Its Way to the Frontier", section "KDA states and MLA KV
 * blocks share one paged pool"), and verifies drafted tokens before it moves a state
 * ("k3_training_and_infra_notes", section 4.5, KDA decoding).  The four calls below are a step of
 * such a decode around kda_decode_window, all on device lengths (a captured graph can be replayed
 * while the lengths change):
 *     kda_paged_plan       lengths -> block tables, token positions, cache slots
 *     kda_paged_append     the step's keys and values into the cache, 8 bits
 *     kda_paged_attention  every run token's attention over its request's pages
 *     kda_verify_draft     accepted drafts and the next token; its `commit` is the argument of
 *                          kda_decode_window
 * A run is a request's new tokens of the step, packed as in kda_decode_window (rows cu_seqlens[n]
 * .. cu_seqlens[n + 1] - 1): one token in a plain decode, what came before and its drafts in a
 * speculative one, a chunk of a prompt in a prefill.  Runs may be empty.
 *
 * The attention is grouped-query over keys and values of 128 channels each; a latent cache (one key
 * head, keys wider than values) is another layout, which these calls do not take.
 *
 * Cache: pages of page_size tokens (16, 32, 64 or 128), the tokens of one head contiguous:
 *     k_cache, v_cache  device e4m3 [num_pages, num_kv_heads, page_size, 128], 16-byte aligned
 *     k_scale, v_scale  device fp32 [num_pages, num_kv_heads], > 0: value = code * scale
 * num_pages * page_size must fit 31 bits (KDA_ERR_UNSUPPORTED); byte offsets are 64-bit.
 * Lengths, tables and slots that point outside what the arguments describe are found on the
 * device: nothing outside is touched and the status word gets KDA_ERR_INVALID_ARG.
 */

/*
 * kda_paged_plan — block tables, positions and slots of a step, in one launch.
 *
 * Request n has cached_lens[n] tokens in the held[n] pages its table row begins with (at least
 * enough pages for them), and its run adds more.  Where its pages do not hold the new total,
 * further ones are taken from the end of the free list, request by request in order.  A request
 * whose demand, added to that of all requests before it, exceeds the list gets no page (nor does
 * one whose total exceeds table_width pages): its tokens' slots are -1 and its lengths stay.  A
 * request that needs no new page is served whatever the others need.
 * release[n] != 0: the request is done.  Its pages are pushed on the end of the free list before
 * any is taken, its table row is free afterwards, and tokens in its run get slot -1.
 *
 *   num_seqs       N, 1 .. 8192 (KDA_ERR_UNSUPPORTED above)
 *   total_tokens   T: rows of positions and slot_map
 *   cached_lens, held  device int32 [N];  cu_seqlens: device int32 [N + 1]
 *   release        device int32 [N], or NULL (none)
 *   block_tables   device int32 [N, table_width]: the entries of new pages are written
 *   free_list      device int32 [free_capacity], free_count (device int32 [1]) entries in use:
 *                  released pages are written after them
 *   context_lens   device int32 [N]: tokens of the request with its run (cached_lens[n] where it is
 *                  not served, 0 where it is released)
 *   held_out, free_count_out   device int32 [N] and [1]: what the next step's call takes as held
 *                  and free_count; not the inputs themselves
 *   positions      device int32 [T]: each token's position in its request
 *   slot_map       device int32 [T]: page * page_size + offset, or -1
 * The inputs other than block_tables and free_list are not written, so the same call repeated
 * gives the same results.
 */
kda_status kda_paged_plan(int32_t num_seqs, int32_t table_width, int32_t page_size,
                          int64_t total_tokens, int32_t free_capacity, const int32_t* cached_lens,
                          const int32_t* cu_seqlens, const int32_t* release, const int32_t* held,
                          int32_t* block_tables, int32_t* free_list, const int32_t* free_count,
                          int32_t* context_lens, int32_t* held_out, int32_t* free_count_out,
                          int32_t* positions, int32_t* slot_map, kda_stream_t stream);

/*
 * kda_paged_append — keys and values of new tokens into their slots, coded in e4m3.
 *
 * The tokens of one call that share a page are consecutive rows, in ascending offsets, and what
 * the page holds below the first of them stays (what lies above is free).  With s_new the smallest
 * power of two >= 2^-100 for which every finite |x| written to the (page, head) is at most 448
 * s_new, the scale becomes s_new in a page whose first token is written by the call and
 * max(s_old, s_new) otherwise; codes are x / scale to the nearest e4m3, ties to even, and codes
 * held before are scaled by s_old / scale and rounded again where the scale grew.  NaN and
 * infinities become NaN and do not count towards the scale.  A NaN s_old stays, and the codes written
 * under it are NaN.
 * A scale only grows until its page is begun anew.  Drafts that are rejected later may have raised
 * it; the tokens that stay then keep the coarser codes (the next step writes over the drafts').
 *
 *   k, v      device bf16 [total_tokens, num_kv_heads, 128]; consecutive tokens k_stride and
 *             v_stride elements apart (a multiple of 8, at least num_kv_heads * 128), so that
 *             slices of a fused projection need no copy; 16-byte aligned
 *   slot_map  device int32 [total_tokens]; a token with a negative slot is not written
 *   num_kv_heads  at most 65535
 */
kda_status kda_paged_append(int64_t total_tokens, int32_t num_kv_heads, int32_t page_size,
                            int32_t num_pages, const void* k, int64_t k_stride, const void* v,
                            int64_t v_stride, const int32_t* slot_map, void* k_cache, void* v_cache,
                            float* k_scale, float* v_scale, kda_stream_t stream);

/*
 * kda_paged_attention — softmax attention of every run token over its request's pages.
 *
 * Run token i of request n, of L_n, attends to its request's keys 0 .. context_lens[n] - L_n + i
 * (the run itself is in the cache already).  Query head h reads key head h / (num_heads /
 * num_kv_heads).  Scores are (q . k) * sm_scale; a token that sees no key gets zeros.
 *
 *   sm_scale      host: finite, > 0
 *   q             device bf16 [total_tokens, num_heads, 128], tokens q_stride elements apart (as
 *                 for kda_paged_append), 16-byte aligned
 *   block_tables  device int32 [num_seqs, table_width]; entries beyond a request's pages are not
 *                 read.  What a page holds beyond its request's context does not matter.
 *   context_lens  device int32 [num_seqs], as from kda_paged_plan
 *   max_run       host: no run is longer (a longer one sets KDA_ERR_INVALID_ARG in the status word)
 *   out           device bf16 [total_tokens, num_heads, 128], contiguous; not q
 *   workspace     device, kda_paged_attention_workspace_bytes(...) bytes, 256-byte aligned.  Its
 *                 size does not depend on the lengths or the number of requests; contents on entry
 *                 are ignored.  Calls that may run at the same time need one each.
 * Scores and sums are fp32 over exact products of the bf16 queries and the cache's values, but for
 * a query's elements below 2^-13 of its largest, which are held within 2^-21 of that largest.
 * Softmax weights meet the values with 11 bits; one below 2^-15 of its row's largest (weight times
 * value scale) is held within 2^-25 of that largest, and equal ones side by side within 2^-29 of it
 * on average, so that a long tail of light weights keeps its sum.
 * num_pages is at least 1 here, num_heads at most 65535; table_width * page_size up to 2^31 - 128 and
 * total_tokens * num_heads up to 2^31 - 256 (KDA_ERR_UNSUPPORTED above).  Rows outside every run are
 * left unwritten.  Results do not depend on the order in which blocks run, so a repeated call gives
 * the same bits; but which contexts are cut between blocks, and which rows share a tile, follows the
 * whole batch, so a request's results may differ in their last bits next to other requests.
 */
size_t kda_paged_attention_workspace_bytes(int32_t num_heads, int32_t num_kv_heads,
                                           int32_t max_run);
kda_status kda_paged_attention(int32_t num_seqs, int64_t total_tokens, int32_t num_heads,
                               int32_t num_kv_heads, int32_t page_size, int32_t num_pages,
                               int32_t table_width, int32_t max_run, float sm_scale, const void* q,
                               int64_t q_stride, const int32_t* cu_seqlens,
                               const int32_t* block_tables, const int32_t* context_lens,
                               const void* k_cache, const void* v_cache, const float* k_scale,
                               const float* v_scale, void* out, void* workspace,
                               size_t workspace_bytes, kda_stream_t stream);

/*
 * kda_verify_draft — which drafted tokens hold, and the token after them.
 *
 * A run of L tokens is the request's last token and L - 1 drafts; the target's probabilities of
 * run row i judge draft x = tokens[row i + 1].  With p and q that row of target_probs and
 * draft_probs and u its uniform number, the draft holds if u * q[x] < p[x] (in fp32).  Drafts hold
 * up to the first that does not, at row a; the next token is then the v with the largest w[v] /
 * e[v], w = max(p - q, 0) of row a, or p itself if that is zero everywhere; where every draft
 * holds, a is the last row and w = p.  Ties go to the lowest v.  With u uniform in [0, 1) and e
 * exponentially distributed, accepted drafts and next token together follow the target's
 * distribution.
 *
 *   target_probs   device [total_tokens, vocab], prob_dtype KDA_FP32 or KDA_BF16
 *   draft_probs    as target_probs (a run's last row is not read), or NULL: drafts are certain,
 *                  q[x] = 1 and 0 elsewhere
 *   tokens         device int32 [total_tokens]: the run tokens
 *   uniform        device fp32 [total_tokens], in [0, 1);  noise: device fp32 [num_seqs, vocab], >= 0
 *   commit         device int32 [num_seqs]: run tokens that stand (the first and the accepted
 *                  drafts; 0 for an empty run)
 *   next_token     device int32 [num_seqs], -1 for an empty run
 *   out_tokens     device int32 [total_tokens]: per run the accepted drafts, the next token, then
 *                  -1; not tokens
 *   num_seqs       at most 65535;  vocab: at most 2^30 (KDA_ERR_UNSUPPORTED above)
 * A draft outside the vocabulary does not hold and sets KDA_ERR_INVALID_ARG in the status word.
 */
kda_status kda_verify_draft(int32_t num_seqs, int64_t total_tokens, int32_t vocab,
                            int32_t prob_dtype, const void* target_probs, const void* draft_probs,
                            const int32_t* tokens, const int32_t* cu_seqlens, const float* uniform,
                            const float* noise, int32_t* commit, int32_t* next_token,
                            int32_t* out_tokens, kda_stream_t stream);

/* ------------------------------------------------------------------ Vocabulary rows
 *
 * Rows of logits x over a vocabulary, KDA_BF16 or KDA_FP32, [total_rows, vocab] with consecutive rows
 * row_stride (>= vocab) elements apart; rows need no alignment beyond their type's.  A row with a NaN
 * or +inf, or without any entry above -inf, has no distribution.  Entries of -inf have probability 0.
 * Exponentials and sums are fp32.
 */

/*
 * kda_token_logprobs — log probabilities of given tokens, entropies, likeliest alternatives.
 *
 * With y = x * inv_temperature and lse = log sum exp(y): logprobs = y[token] - lse, entropy = -sum p
 * log p with p = exp(y - lse) in nats, and the top_k largest x in falling order, the lowest index
 * first among equals, with their y - lse.
 *
 *   tokens           device int32 [total_rows], or NULL: none asked for, logprobs is not written.  A
 *                    row whose token is negative is skipped: 0, 0, and no alternatives.  A token >=
 *                    vocab counts as negative and sets KDA_ERR_INVALID_ARG in the status word.
 *   inv_temperature  device fp32 [total_rows], above 0 and at most 2^127, or NULL: ones
 *   top_k            0 .. 128 (KDA_ERR_UNSUPPORTED above)
 *   logprobs, entropy          device fp32 [total_rows]
 *   top_ids, top_logprobs      device int32 and fp32 [total_rows, top_k] (not used for top_k 0).
 *                    Entries of -inf are no alternatives: where fewer than top_k are left, -1 and -inf.
 *   vocab            at most 2^30 (KDA_ERR_UNSUPPORTED above)
 * A row without a distribution, or whose inv_temperature is not in that range, gets NaN and -1.
 */
kda_status kda_token_logprobs(int64_t total_rows, int32_t vocab, int32_t logit_dtype,
                              const void* logits, int64_t row_stride, const int32_t* tokens,
                              const float* inv_temperature, int32_t top_k, float* logprobs,
                              float* entropy, int32_t* top_ids, float* top_logprobs,
                              kda_stream_t stream);

/*
 * kda_distill_topk — Kullback-Leibler divergence of the rows from a teacher's top entries.
 *
 * With q = softmax(x * inv_temperature) and a row's entries (id_i, v_i):
 *   tail == 0:  p = softmax(v) over the entries;  loss = sum_i p_i (log p_i - log q[id_i])
 *   tail == 1:  v are log probabilities, p_i = exp(v_i), r = max(0, 1 - sum p); with q_r the mass of
 *               the tokens that no entry names, loss = the same sum + r (log r - log q_r)
 * Terms with p_i = 0 or r = 0 are 0.  An entry with a negative id is absent; one >= vocab is too, and
 * sets KDA_ERR_INVALID_ARG in the status word.  Entries may name a token more than once.  A row
 * without entries (with tail == 0: without one above -inf) is skipped; its loss is 0.
 *
 *   num_teacher      1 .. 256 entries a row (KDA_ERR_UNSUPPORTED above); with tail less than vocab
 *   teacher_ids, teacher_values   device int32 and fp32 [total_rows, num_teacher]
 *   inv_temperature  host: > 0, at most 1e30.  The values are taken at the temperature that they have.
 *   loss             device fp32 [total_rows]
 *   stats            device fp32 [total_rows, 4], 16-byte aligned, for kda_distill_topk_bwd: the
 *                    largest x and the sum of exp((x - it) * inv_temperature), and the same over the
 *                    tokens that no entry names; zeros for a row that is skipped
 *   vocab            at most 786,432 entries in bf16, 393,216 in fp32 (KDA_ERR_UNSUPPORTED above)
 * A row without a distribution has loss NaN.  Repeated calls give the same bits.
 */
kda_status kda_distill_topk(int64_t total_rows, int32_t vocab, int32_t logit_dtype,
                            const void* logits, int64_t row_stride, int32_t num_teacher,
                            const int32_t* teacher_ids, const float* teacher_values,
                            float inv_temperature, int32_t tail, float* loss, float* stats,
                            kda_stream_t stream);

/*
 * kda_distill_topk_bwd — d_logits = d_loss times the gradient of kda_distill_topk's losses:
 * inv_temperature * (M q_v - sum of the p_i of token v), M = sum p (+ r with tail), and for the tokens
 * that no entry names - inv_temperature * r q_v / q_r besides.
 *
 *   stats     as kda_distill_topk wrote it for the same inputs
 *   d_loss    device fp32 [total_rows]; a row with 0 (or without entries) is skipped and gets zeros
 *   d_logits  device [total_rows, vocab] of the logits' type, rows d_row_stride elements apart; it may
 *             be logits with the same stride, and must not overlap it otherwise.  Rows of both that
 *             are equally far from 16-byte boundaries are faster: vectors need no shifting.
 * Where the tokens that no entry names have no mass at all, r's share of the gradient is left out.
 */
kda_status kda_distill_topk_bwd(int64_t total_rows, int32_t vocab, int32_t logit_dtype,
                                const void* logits, int64_t row_stride, int32_t num_teacher,
                                const int32_t* teacher_ids, const float* teacher_values,
                                float inv_temperature, int32_t tail, const float* stats,
                                const float* d_loss, void* d_logits, int64_t d_row_stride,
                                kda_stream_t stream);

/*
 * kda_distill_topk_grad — kda_distill_topk's losses and d_logits for sum(weight * loss).  Rows are
 * read twice, the second time mostly from L2.  loss is not multiplied by weight.  A row without
 * entries gets loss 0 and zeros, one with weight 0 its loss and zeros, whatever its logits are.
 * Arguments as above.
 */
kda_status kda_distill_topk_grad(int64_t total_rows, int32_t vocab, int32_t logit_dtype,
                                 const void* logits, int64_t row_stride, int32_t num_teacher,
                                 const int32_t* teacher_ids, const float* teacher_values,
                                 float inv_temperature, int32_t tail, const float* weight,
                                 float* loss, void* d_logits, int64_t d_row_stride,
                                 kda_stream_t stream);

/*
 * kda_selftest_wait_timeout — diagnostic: launch one CTA that waits, through the kernels' own
 * bounded-wait code, on a barrier phase nothing completes.  The wait gives up after its limit
 * (about 2 s) and records KDA_ERR_TIMEOUT in the sticky status word, which
 * kda_read_device_status() then returns; the context stays usable.  Every wait of the compute
 * kernels is bounded the same way, so a lost arrival (a defect, or a fault elsewhere) ends as a
 * status code rather than a hang.  Returns KDA_OK once launched.
 */
kda_status kda_selftest_wait_timeout(kda_stream_t stream);

/*
 * kda_read_device_status — synchronise `stream`, then return and clear the sticky device
 * status word of the current device (KDA_OK when no kernel reported a problem).
 */
kda_status kda_read_device_status(kda_stream_t stream);

/* Human-readable name of a status code (static string). */
const char* kda_status_string(kda_status status);

/* Number of kernels this library has launched in this process (all devices, all streams). */
uint64_t kda_launch_count(void);

/* Library ABI version (increments on any signature change). */
int32_t kda_version(void);

#ifdef __cplusplus
}
#endif

#endif /* KDA_GB300_H */
