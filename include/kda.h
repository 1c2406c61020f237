/*
 * kda.h -- C ABI of libkda.so: the Kimi Delta Attention (KDA) operator on
 * one NVIDIA GB300 GPU (sm_103a).
 *
 * The operator, per sequence and head, carries a d_k x d_v fp32 state S
 * (row i = key channel, column j = value channel) through
 *
 *     S_t = (I - beta_t k_t k_t^T) Diag(exp(g_t)) S_{t-1} + beta_t k_t v_t^T
 *     o_t = scale * S_t^T q_t
 *
 * i.e. per token: forget (per-channel decay), correct (delta-rule erase of
 * the stale association S^T k - v), write. Sources: "K3 vs DSV4
 * architecture divergence" (locsic.com), KDA section (forget -> correct ->
 * write) and section "硬件适配" (hardware adaptation: log-decay lower bound
 * g_min = -5, so the cumulative decay over a 16-token tile is >= -80 and its
 * reciprocal fits bf16); "Kimi K3: The Manos, The Mythos, The Legendos"
 * (SemiAnalysis), sections "DeltaNet", "Gated DeltaNet" (KDA: diagonal,
 * per-channel forget gate) and "FlashKDA 算法" (chunked prefill with a UT
 * transform; decode follows the per-token form).
 *
 * The library clamps every g to [-5, 0] on load; exp is the natural
 * exponential.
 *
 * Conventions for every entry point:
 *  - All tensor pointers are DEVICE pointers owned by the caller. The library
 *    allocates and frees nothing.
 *  - Calls are asynchronous on `stream` (a cudaStream_t; NULL = the legacy
 *    default stream). The return value reports argument validation and
 *    launch errors only. Errors detected on the device (malformed
 *    cu_seqlens) are recorded in the workspace and read by
 *    kda_workspace_status().
 *  - Dtype codes: KDA_BF16 = 0, KDA_F32 = 1. They select the type of q, k,
 *    v, beta and out. g, the states and the arithmetic are always fp32.
 *  - Return codes are kda_status values.
 *  - Head dimension: d_k = d_v = D = 128 only (KDA_ERR_UNSUPPORTED else).
 */
#ifndef KDA_H
#define KDA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    KDA_OK = 0,
    KDA_ERR_INVALID_ARG = 1, /* null pointer, negative size, bad alignment, size overflow */
    KDA_ERR_UNSUPPORTED = 2, /* D != 128, unsupported chunk or dtype */
    KDA_ERR_CUDA = 3,        /* a CUDA launch or runtime call failed */
    KDA_ERR_TIMEOUT = 4,     /* a bounded device-side wait ran out */
    KDA_ERR_DEVICE = 5,      /* the device flagged bad input (e.g. cu_seqlens) */
    KDA_ERR_TOO_LARGE = 6,   /* kda_prefill_noalloc: the sizes need more scratch than its
                                static array holds */
    KDA_ERR_RANGE = 7,       /* a bf16 prefill state came out non-finite (inputs outside the
                                range that kda_prefill states) */
    KDA_ERR_NO_SPACE = 8     /* a cache call needed more pages than were free */
} kda_status;

typedef enum { KDA_BF16 = 0, KDA_F32 = 1 } kda_dtype;

typedef enum {
    KDA_SCHEDULE_SPLIT = 0,  /* bf16: chunk preparation, then the recurrence */
    KDA_SCHEDULE_FUSED = 1,  /* bf16: both in one cooperative launch */
    KDA_SCHEDULE_DIRECT = 2  /* fp32 I/O: one kernel */
} kda_schedule;

/* Human-readable name of a status code (static string, never NULL). */
const char *kda_status_string(int status);

/* ABI version of this header (major * 100 + minor): 101. */
int kda_abi_version(void);

/*
 * Bytes of device workspace for kda_prefill's fastest plan at these sizes
 * (same meaning as in kda_prefill; varlen != 0 when cu_seqlens will be passed,
 * and then T is the packed total). Returns 0 when the sizes are invalid. The
 * workspace holds the device status word, the chunk schedule and, for bf16
 * I/O, one 74,368-byte prepared block per (chunk, head) plus (fused schedule)
 * one ready flag per block: it grows with the number of tokens. It must be
 * 256-byte aligned and must not be shared by calls in flight at the same time.
 *
 * kda_prefill accepts any workspace of at least kda_prefill_workspace_size_min
 * bytes and runs the fastest plan that it holds (kda_prefill_plan reports
 * which):
 *  - at least kda_prefill_workspace_size: the fastest plan;
 *  - else, at least kda_prefill_workspace_size_ring: the fused schedule with
 *    its blocks in a ring of up to 16 per chain, chains in groups of the
 *    modelled best size, one cooperative launch per group. Its size depends on
 *    the number of chains in a group, not on the sequence lengths (about
 *    35 MB for a group of 29 chains);
 *  - else the same with fewer chains per group (the most that fit), down to
 *    one chain (kda_prefill_workspace_size_min, about 1.2 MB) -- slower.
 * All plans give bit-identical results. fp32 I/O needs 256 bytes.
 */
size_t kda_prefill_workspace_size(int32_t N, int32_t T, int32_t H, int32_t D, int32_t chunk,
                                  int32_t io, int32_t varlen);
size_t kda_prefill_workspace_size_ring(int32_t N, int32_t T, int32_t H, int32_t D, int32_t chunk,
                                       int32_t io, int32_t varlen);
size_t kda_prefill_workspace_size_min(int32_t N, int32_t T, int32_t H, int32_t D, int32_t chunk,
                                      int32_t io, int32_t varlen);

/* The plan that kda_prefill runs for these sizes and workspace size. */
typedef struct {
    int32_t schedule;     /* kda_schedule */
    int32_t groups;       /* fused: cooperative launches, one per group of chains */
    int32_t group_chains; /* fused: (sequence, head) chains per group */
    int32_t ring;         /* fused: prepared blocks per chain in its ring; 0 = one per chunk */
    size_t bytes;         /* workspace bytes that the plan uses */
    int64_t lead_items;   /* fused: blocks prepared on every SM by a launch of producers only
                             before the chains start (0: the chains start at once) */
} kda_prefill_plan_info;

/*
 * Writes to *plan the plan that kda_prefill runs for these sizes (as in
 * kda_prefill_workspace_size) with a workspace of workspace_bytes bytes on the
 * current device. Returns KDA_OK; KDA_ERR_INVALID_ARG when the sizes are
 * invalid, plan is NULL or the workspace is below the minimum; KDA_ERR_CUDA
 * when the device cannot be queried.
 */
int kda_prefill_plan(int32_t N, int32_t T, int32_t H, int32_t D, int32_t chunk, int32_t io,
                     int32_t varlen, size_t workspace_bytes, kda_prefill_plan_info *plan);

/*
 * Chunked-parallel KDA prefill over N sequences.
 *
 * Layout (row-major, contiguous):
 *   q, k : io dtype [T_total, H, D]      v, out : io dtype [T_total, H, D]
 *   g    : fp32     [T_total, H, D]      beta   : io dtype [T_total, H]
 *   init_state, final_state : fp32 [N, H, D(key), D(value)]
 * Sequences:
 *   cu_seqlens == NULL : N sequences of equal length T, stored one after the
 *                        other (T_total = N * T).
 *   cu_seqlens != NULL : DEVICE int32 [N+1] prefix offsets of N packed
 *                        sequences, cu[0] = 0, non-decreasing, cu[N] = T =
 *                        T_total. A length-0 sequence produces no output and
 *                        its final state equals its initial state. Malformed
 *                        offsets are detected on the device: the affected
 *                        sequences are skipped and kda_workspace_status()
 *                        returns KDA_ERR_DEVICE.
 * init_state may be NULL (zero initial state). final_state may be NULL (not
 * written) and may alias init_state (in-place checkpoint update).
 * chunk: tokens per chunk, 64 (bf16 or fp32 I/O) or 16 (fp32 I/O). The
 * result does not depend on the chunk size beyond rounding.
 * scale: multiplies the readout (e.g. 1/sqrt(D)).
 * workspace: device buffer of at least kda_prefill_workspace_size_min()
 * bytes, 256-byte aligned; the plan depends on its size (see
 * kda_prefill_workspace_size). Each call clears its status word on the stream
 * before the kernels run.
 * Pointer alignment: q, k, v, out 16 bytes; g, states 16 bytes.
 * Range (bf16 I/O): the chunk products that involve keys and queries (their
 * Gram matrices) run in bf16; the state path (beta v, the pseudo-values, U and
 * a copy of the state) runs in fp16 for its longer significand, with a
 * power-of-two scale per chunk for beta v and per value column for the state,
 * so any magnitude of v and of the initial state up to about 1e20 is handled,
 * including changes by many orders of magnitude along a sequence. Keys and
 * queries enter fp16 after the decay weights (k e^{-a}, q e^{a} <= 1 per
 * factor): their entries and the products |q||k| must stay well below 6e4, as
 * they do for the L2-normalised keys and queries of a KDA layer. If an fp16
 * value overflows anyway, the final state comes out non-finite and
 * kda_workspace_status() reports KDA_ERR_RANGE (never silently).
 * Accuracy (bf16 I/O): outputs and final states within 2e-2 of an fp64
 * recurrence (largest error / RMS) on the workloads tested; inputs whose
 * chunks repeat one key with beta = 1 and almost no decay reach 2.5-4e-2 (the
 * shared fp16 rounding of the UT inverse's subdiagonal, on rank-one results).
 * Returns KDA_OK after enqueueing the work on `stream`.
 */
int kda_prefill(const void *q, const void *k, const void *v, const float *g, const void *beta,
                float scale, const float *init_state, const int32_t *cu_seqlens, int32_t N,
                int32_t T, int32_t H, int32_t D, int32_t chunk, int32_t io, void *out,
                float *final_state, void *workspace, size_t workspace_bytes, void *stream);

/*
 * kda_prefill with two options (kda_prefill is this with g_per_channel = 1 and
 * snapshot_interval = 0):
 *   g_per_channel : 1 = g fp32 [T_total, H, D] (KDA's channel-wise decay);
 *                   0 = g fp32 [T_total, H], one decay per token and head (the
 *                   Gated DeltaNet form, "K3 vs DSV4 architecture divergence",
 *                   section KDA), clamped to [-5, 0] like the channel-wise one.
 *   snapshot_interval : 0 = none; else a positive multiple of `chunk`: the state
 *                   after every snapshot_interval tokens of each sequence (for
 *                   prefix caching of long prompts) is written to
 *                   snapshots fp32 [N, max_snapshots, H, D, D] (16-byte aligned):
 *                   entry [n][s] = the state after (s + 1) * snapshot_interval
 *                   tokens of sequence n, for s < max_snapshots; entries past a
 *                   sequence's end are not written. The final state of each
 *                   sequence still goes to final_state.
 * Returns KDA_ERR_UNSUPPORTED when snapshot_interval is not a multiple of chunk.
 */
int kda_prefill_ex(const void *q, const void *k, const void *v, const float *g,
                   const void *beta, float scale, const float *init_state,
                   const int32_t *cu_seqlens, int32_t N, int32_t T, int32_t H, int32_t D,
                   int32_t chunk, int32_t io, int32_t g_per_channel, int32_t snapshot_interval,
                   int32_t max_snapshots, float *snapshots, void *out, float *final_state,
                   void *workspace, size_t workspace_bytes, void *stream);

/*
 * One decode step (kda_decode with T = 1, channel-wise g, no indices): B
 * sequences x H heads, one new token each, following the per-token form ("FlashKDA 算法": decode follows the recurrence; its cost
 * is dominated by one fp32 read and one fp32 write of the state, ~8 D^2
 * bytes per head and token, "复杂度分析").
 *   q, k, v : io dtype [B, H, D]   g : fp32 [B, H, D]   beta : io dtype [B, H]
 *   state_inout : fp32 [B, H, D, D], updated in place
 *   out : io dtype [B, H, D]
 * Pointer alignment: 16 bytes. Needs no workspace.
 */
int kda_decode_step(const void *q, const void *k, const void *v, const float *g,
                    const void *beta, float scale, int32_t B, int32_t H, int32_t D, int32_t io,
                    float *state_inout, void *out, void *stream);

/*
 * Kernel schedule that kda_prefill uses for these sizes on the current device
 * with a workspace of kda_prefill_workspace_size bytes (arguments as in
 * kda_prefill_workspace_size):
 *   KDA_SCHEDULE_SPLIT  bf16: the chunk-preparation kernel over all
 *                       (chunk, head) blocks, then the recurrence kernel,
 *                       one CTA per (sequence, head) chain;
 *   KDA_SCHEDULE_FUSED  bf16: one cooperative launch in which one CTA per
 *                       chain runs the recurrence while the other SMs prepare
 *                       blocks in chunk order, chains waiting (bounded) on a
 *                       per-block ready flag; chosen when the chains take at
 *                       most a third of the SMs, and with more chains (up to
 *                       the SMs less 16) when a lead launch first prepares
 *                       the leading blocks on every SM, so that the chains
 *                       then never wait for the other SMs' blocks, is
 *                       modelled at least 3 % faster than the split schedule
 *                       (kda_prefill_plan_info.lead_items);
 *   KDA_SCHEDULE_DIRECT fp32 I/O: one kernel on CUDA cores.
 * With cu_seqlens a schedule kernel runs first. kda_prefill_set_schedule
 * overrides the bf16 choice. Returns the schedule, or the negated kda_status
 * on invalid sizes or a failed device query. The result does not depend on
 * the schedule: both bf16 schedules run the same arithmetic.
 */
int kda_prefill_schedule(int32_t N, int32_t T, int32_t H, int32_t D, int32_t chunk, int32_t io,
                         int32_t varlen);

/*
 * Process-wide override of the bf16 prefill schedule, for tuning and for tests
 * that run both schedules on the same inputs: -1 = the automatic choice (the
 * default), KDA_SCHEDULE_SPLIT or KDA_SCHEDULE_FUSED ("fused" still needs
 * fewer chains than SMs). When the library is loaded the environment variable
 * KDA_PREFILL_SCHEDULE=split|fused sets the initial value; it is not read
 * again. Calls already enqueued are not affected. Returns the previous value,
 * or -KDA_ERR_INVALID_ARG for any other argument.
 */
int kda_prefill_set_schedule(int schedule);

/*
 * Decode of T new tokens for each of B sequences (T = 1: one step; T up to 64,
 * e.g. the drafted tokens of speculative decoding), the per-token recurrence
 * applied in order, with each head's state read once and written once
 * ("FlashKDA 算法", "复杂度分析": ~8 D^2 bytes of state traffic per head and step).
 *   q, k, v : io dtype [B, T, H, D]   beta : io dtype [B, T, H]
 *   g       : fp32 [B, T, H, D] when g_per_channel = 1 (KDA), or fp32 [B, T, H]
 *             when g_per_channel = 0 (one decay per token and head: the Gated
 *             DeltaNet form; clamped to [-5, 0] like the channel-wise one)
 *   state_pool : fp32 [pool_size, H, D, D], updated in place
 *   state_indices : DEVICE int32 [B], the pool entry of each sequence, or NULL
 *             (sequence b uses entry b; then pool_size >= B). An index < 0 or
 *             >= pool_size skips its sequence (no output, no state change).
 *             Indices must be distinct among the sequences of one call: two
 *             sequences on one entry update it concurrently, and the entry
 *             and both outputs are then undefined (not detected).
 *   out : io dtype [B, T, H, D]; must not alias the inputs or the pool.
 * Pointer alignment: 16 bytes (q, k, v, out, the pool; g when per channel).
 * Needs no workspace. T = 0 or B = 0 is a no-op.
 * Returns KDA_ERR_UNSUPPORTED for T > 64, D != 128 or an unknown io.
 */
int kda_decode(const void *q, const void *k, const void *v, const float *g, const void *beta,
               float scale, int32_t B, int32_t T, int32_t H, int32_t D, int32_t io,
               int32_t g_per_channel, float *state_pool, int32_t pool_size,
               const int32_t *state_indices, void *out, void *stream);

/*
 * The layer steps on either side of the operator ("Kimi K3: The Manos, The
 * Mythos, The Legendos", section "Kimi Linear"); the projections themselves are
 * plain matrix products done by the caller. Rows are [T_total, H, D], D = 128.
 *
 * kda_layer_prologue: from the projected q_raw, k_raw, v_raw, alpha_raw (io
 * dtype [T_total, H, D]) and beta_raw (io dtype [T_total, H]):
 *   q = l2(conv(q_raw)), k = l2(conv(k_raw)), v = conv(v_raw),
 *   g = -5 sigmoid(alpha_raw) (fp32 [T_total, H, D]), beta = sigmoid(beta_raw),
 * where conv is a depthwise causal convolution of width W (1..4) along each
 * sequence, left-padded with zeros (weights conv_* fp32 [H, D, W]; tap W - 1
 * multiplies the current token), with no activation, and l2(x) = x /
 * sqrt(sum x^2 + 1e-6) over the D channels of a (token, head). cu_seqlens:
 * DEVICE int32 [N + 1] offsets of packed sequences (NULL: one sequence);
 * convolutions never cross a sequence start. Outputs may not alias inputs.
 * Pointer alignment: 8 bytes (bf16) or 16 bytes (fp32) for the [.., D] rows,
 * 16 bytes for g and for the conv weights; a misaligned pointer returns
 * KDA_ERR_INVALID_ARG before any launch.
 *
 * kda_layer_epilogue: y = o / sqrt(mean(o^2) + 1e-6) * w * sigmoid(gate_raw)
 * per (token, head) over its D channels: o, gate_raw, y io dtype
 * [T_total, H, D], 16-byte aligned (both dtypes); norm_weight fp32 [D]
 * (16-byte aligned).
 *
 * Both return KDA_ERR_UNSUPPORTED for D != 128, W outside 1..4 or an unknown
 * io; T_total = 0 is a no-op.
 */
int kda_layer_prologue(const void *q_raw, const void *k_raw, const void *v_raw,
                       const void *alpha_raw, const void *beta_raw, const float *conv_q,
                       const float *conv_k, const float *conv_v, int32_t W,
                       const int32_t *cu_seqlens, int32_t N, int32_t T_total, int32_t H, int32_t D,
                       int32_t io, void *q, void *k, void *v, float *g, void *beta, void *stream);
int kda_layer_epilogue(const void *o, const void *gate_raw, const float *norm_weight,
                       int32_t T_total, int32_t H, int32_t D, int32_t io, void *y, void *stream);

/*
 * kda_layer_prologue at decode time: T new tokens for each of B sequences,
 * with the short convolutions' windows carried between calls ("Kimi Linear":
 * the convolution applies to every token, so a decoding sequence keeps the
 * last W - 1 projected inputs of q, k and v).
 *   q_raw, k_raw, v_raw, alpha_raw : io dtype [B, T, H, D]   beta_raw : io dtype [B, T, H]
 *   conv_state : io dtype [pool_size, 3 (q, k, v), W - 1, H, D], updated in place:
 *                row r of an entry is the raw input W - 1 - r tokens back (the
 *                most recent last). A new sequence starts from zeros (the left
 *                padding of kda_layer_prologue); after a prompt of length L, rows
 *                hold the prompt's raw inputs L - W + 1 .. L - 1 (zeros before 0).
 *                May be NULL when W = 1.
 *   state_indices : DEVICE int32 [B], the pool entry of each sequence, or NULL
 *                (sequence b uses entry b); an index < 0 or >= pool_size skips
 *                its sequence (nothing written). Indices must be distinct.
 *   outputs q, k, v : io dtype [B, T, H, D]; g : fp32 [B, T, H, D]; beta : io dtype [B, T, H]
 * Weights, arithmetic, alignment and return codes as kda_layer_prologue (the
 * conv_state rows like the [.., D] rows). B = 0 or T = 0 is a no-op.
 */
int kda_layer_prologue_decode(const void *q_raw, const void *k_raw, const void *v_raw,
                              const void *alpha_raw, const void *beta_raw, const float *conv_q,
                              const float *conv_k, const float *conv_v, int32_t W, int32_t B,
                              int32_t T, int32_t H, int32_t D, int32_t io, void *conv_state,
                              int32_t pool_size, const int32_t *state_indices, void *q, void *k,
                              void *v, float *g, void *beta, void *stream);

/*
 * Synchronises `stream`, then reads and clears the device status word of a
 * kda_prefill, kda_attn_* or kda_cache_* workspace. Returns KDA_OK,
 * KDA_ERR_TIMEOUT, KDA_ERR_DEVICE (malformed cu_seqlens, lengths, rows or page
 * numbers were seen), KDA_ERR_RANGE (a final state of the bf16 path was not
 * finite), KDA_ERR_NO_SPACE or KDA_ERR_CUDA, the first that applies in this
 * order.
 */
int kda_workspace_status(void *workspace, void *stream);

/*
 * Host-side check of a HOST copy of cu_seqlens (N+1 int32): cu[0] = 0,
 * non-decreasing, cu[N] = T_total. Returns KDA_OK or KDA_ERR_INVALID_ARG.
 */
int kda_check_cu_seqlens(const int32_t *cu_seqlens_host, int32_t N, int32_t T_total);

/*
 * kda_prefill_noalloc -- the same prefill as kda_prefill, for callers that
 * cannot allocate device memory (no access to cudaMalloc or to the host
 * framework's allocator, or code that must not allocate at the point of the
 * call). It takes no workspace: its scratch is a static device array inside
 * the library, 16 MiB on every GPU that loads the library, held until the
 * process exits. The pages have no counterpart to this entry point; it exists
 * for such callers only.
 *  - Arguments, layouts, stream semantics and results are those of
 *    kda_prefill without the workspace arguments.
 *  - It runs the plan that a 16 MiB workspace gets (kda_prefill_plan with
 *    workspace_bytes = 16 MiB): the fastest one while it fits, else the
 *    fused schedule with rings. Sizes whose kda_prefill_workspace_size_min()
 *    exceeds 16 MiB (only packed batches of about two million sequences) are
 *    rejected with KDA_ERR_TOO_LARGE; nothing is launched.
 *  - The first call on a device (with that device current) looks up the
 *    array's device address; make that first call before any stream capture.
 *  - All calls share the one array and each call clears its status word
 *    first: calls that overlap on the GPU race on it, so the caller must
 *    serialise them (one stream, or events between streams).
 *  - Errors found on the device (malformed cu_seqlens, a timed-out wait) are
 *    recorded in the array's status word; read them with kda_noalloc_status().
 *  - It allocates nothing (no cudaMalloc / cudaFree, no allocating library
 *    routine).
 */
int kda_prefill_noalloc(const void *q, const void *k, const void *v, const float *g,
                        const void *beta, float scale, const float *init_state,
                        const int32_t *cu_seqlens, int32_t N, int32_t T, int32_t H, int32_t D,
                        int32_t chunk, int32_t io, void *out, float *final_state, void *stream);

/*
 * The device status word of kda_prefill_noalloc's static array on the current
 * device (the counterpart of kda_workspace_status for that entry point; the
 * pages have no counterpart either): synchronises `stream`, then reads and
 * clears the word. It reports the device-side errors of the noalloc calls
 * since the last read (each call clears the word before its kernels run, so
 * normally those of the last call): KDA_OK, KDA_ERR_DEVICE (malformed
 * cu_seqlens), KDA_ERR_TIMEOUT, or KDA_ERR_CUDA if a CUDA call failed. Like
 * the entry point itself it allocates nothing; make the first call on a
 * device before any stream capture.
 */
int kda_noalloc_status(void *stream);

/*
 * Softmax attention, for the full-attention layers that stand between a model's
 * KDA layers ("K3 vs DSV4 architecture divergence", KDA section: the layers
 * alternate; there with gated MLA, whose cache of one latent row per token these
 * calls do not read: they take K and V heads of 128 channels). Hq query heads share Hkv key/value heads, G = Hq / Hkv <= 64 each:
 *
 *     o_i = sum_j p_ij v_j / sum_j p_ij,   p_ij = exp(scale q_i . k_j),
 *     lse_i = ln sum_j p_ij,
 *
 * over the keys j that row i sees; a row that sees none has o = 0 and
 * lse = -inf. Logits, maxima and sums are fp32 (with bf16 I/O p is rounded to
 * bf16 for the product with v, out to bf16 at the end). A sequence's keys only
 * ever touch its own rows: whatever lies past a sequence's end (another
 * sequence, the rest of a page, NaN) is not used. Inside a sequence a NaN or an infinity
 * in v also reaches, in its channel, rows that do not see it but share its key tile (128 keys,
 * fp32 64; a call's drafts are a tile), as 0 * NaN and 0 * infinity do.
 * scale: finite and > 0. D = 128.
 *
 * Workspace: device buffer, 256-byte aligned, of the size that the query gives
 * (it holds the status word and the parts of rows that several SMs share). Its
 * first 256 bytes must be zero before its first use; calls do not clear the
 * status word, kda_workspace_status() reads and clears it. It must not be shared
 * by calls in flight at the same time.
 *
 * kda_attn_prefill: causal attention over N packed sequences.
 *   q    : io dtype [Tq_total, Hq, D], ldq elements from one token to the next
 *   k, v : io dtype [Tk_total, Hkv, D], ldk and ldv likewise (so that q, k and v
 *          may be views of one projection's rows)
 *   out  : io dtype [Tq_total, Hq, D], contiguous   lse : fp32 [Tq_total, Hq] or NULL
 *   cu_seqlens_q, cu_seqlens_k : DEVICE int32 [N + 1] offsets, each from 0, non-decreasing, to
 *          at most the total (then Tq and Tk are the totals). cu_seqlens_k NULL with
 *          cu_seqlens_q given: the keys have the same offsets (Tk = Tq). Both NULL:
 *          equal lengths Tq and Tk (the totals are N Tq and N Tk).
 *   Token i of a sequence with Lq tokens and Lk keys sees the keys j <= i + Lk - Lq:
 *   Lk = Lq is a prompt, Lk > Lq tokens appended to a prefix whose keys come
 *   first; with Lk < Lq the first Lq - Lk tokens see nothing.
 *   Malformed offsets are flagged on the device (KDA_ERR_DEVICE from
 *   kda_workspace_status) and the whole call is skipped.
 * Pointers 16-byte aligned; ldq >= Hq D, ldk, ldv >= Hkv D, each a multiple of 16 bytes.
 * Returns KDA_ERR_UNSUPPORTED for D != 128, G > 64 or an unknown io; N = 0 or no
 * token is a no-op.
 */
size_t kda_attn_prefill_workspace_size(int32_t N, int32_t Tq_total, int32_t Tk_total, int32_t Hq,
                                       int32_t Hkv, int32_t D, int32_t io);
int kda_attn_prefill(const void *q, const void *k, const void *v, int64_t ldq, int64_t ldk,
                     int64_t ldv, float scale, const int32_t *cu_seqlens_q,
                     const int32_t *cu_seqlens_k, int32_t N, int32_t Tq, int32_t Tk, int32_t Hq,
                     int32_t Hkv, int32_t D, int32_t io, void *out, float *lse, void *workspace,
                     size_t workspace_bytes, void *stream);

/*
 * kda_attn_decode: attention of T new tokens (1..64) of each of B sequences over
 * a paged cache and over one another: T = 1 is the plain decode step, T > 1 the
 * drafted tokens of speculative decoding, as a chain or a tree.
 *   q : io dtype [B, T, Hq, D], ldq elements from one token to the next (a
 *       sequence's tokens are T ldq apart)
 *   k_pages, v_pages : io dtype [num_pages, Hkv, page_size, D]; page_size 16, 32, 64,
 *       128 or 256
 *   block_table : DEVICE int32 [B, table_cols], row b's pages in order, table_ld
 *       entries from one row to the next
 *   seq_lens : DEVICE int32 [B], tokens of each sequence in the cache (0 is fine)
 *   k_new, v_new : io dtype [B, T, Hkv, D] (ldk, ldv), the new tokens' own keys and
 *       values, not (yet) in the cache; both NULL: the tokens see the cache alone
 *   tree_mask : DEVICE uint64 [B, T] or NULL. Bit s of [b][t]: new token t sees new
 *       token s (its ancestors in the tree and itself). NULL: the chain, s <= t.
 *   out : io dtype [B, T, Hq, D], contiguous   lse : fp32 [B, T, Hq] or NULL
 * Every token sees all seq_lens[b] cached ones. A length outside
 * 0..table_cols page_size is flagged (KDA_ERR_DEVICE) and its sequence skipped
 * (nothing written); a page number outside the pool is flagged and its keys read
 * as zeros. table_cols page_size may be 2^31 - 1024 at most. kda_cache_append adds
 * the accepted tokens to the cache.
 * Workspace, alignment and errors as kda_attn_prefill; T > 64 or another page size
 * is KDA_ERR_UNSUPPORTED. B = 0 or T = 0 is a no-op.
 */
size_t kda_attn_decode_workspace_size(int32_t B, int32_t T, int32_t Hq, int32_t Hkv, int32_t D,
                                      int32_t page_size, int32_t table_cols, int32_t io);
int kda_attn_decode(const void *q, int64_t ldq, const void *k_new, const void *v_new, int64_t ldk,
                    int64_t ldv, const void *k_pages, const void *v_pages, int32_t num_pages,
                    int32_t page_size, const int32_t *block_table, int64_t table_ld,
                    int32_t table_cols, const int32_t *seq_lens, const uint64_t *tree_mask,
                    float scale, int32_t B, int32_t T, int32_t Hq, int32_t Hkv, int32_t D,
                    int32_t io, void *out, float *lse, void *workspace, size_t workspace_bytes,
                    void *stream);

/*
 * The pages of a cache. block_table int32 [rows, table_cols] (table_ld entries
 * from one row to the next): a row's pages in order, then -1; seq_lens int32
 * [rows]; refs int32 [num_pages] (16-byte aligned): the table entries on each page,
 * 0 = free. All three are DEVICE arrays that these calls update, for any number of
 * layers' pools at once. num_pages and rows * table_cols are at most 2^31 - 2^16. Pages
 * are chosen lowest number first, so results depend on the inputs alone. `workspace` (256-byte aligned, kda_cache_workspace_size
 * bytes, its first 256 bytes zero before its first use) also takes the status:
 * malformed rows, lengths or page numbers are skipped and flagged
 * (KDA_ERR_DEVICE); a call that needs more pages than are free changes nothing
 * and is flagged (KDA_ERR_NO_SPACE).
 *
 * kda_cache_alloc: gives every row the pages it lacks for want[row] tokens (DEVICE
 *   int32 [rows]; a row never loses pages). seq_lens is not touched.
 * kda_cache_fork: for i < n, row dst[i] (which must be empty, else it is flagged and
 *   skipped) becomes a copy of row src[i]: full pages are shared (refs + 1); where
 *   the length ends inside a page, dst gets a fresh page, and copies[i] = (shared
 *   page, fresh page) has to be copied in every pool (kda_cache_copy); copies[i] =
 *   (-1, -1) otherwise. A src whose length ends inside a page that is not in the
 *   pool is flagged and its pair skipped: dst stays empty and takes no page. src or
 *   dst < 0 skips the pair. No dst may be another pair's src or dst.
 * kda_cache_free: drops the pages of rows[i], i < n (distinct; < 0 is skipped): refs - 1,
 *   entries -1, length 0.
 * kda_cache_compact: with L live pages, the j-th live page numbered >= L moves to
 *   the j-th free page below L; table entries are renamed, refs moved; copies
 *   int32 [num_pages, 2] gets the (from, to) pairs, then (-1, -1); *count (DEVICE) their
 *   number. Afterwards the live pages are 0 .. L - 1.
 * kda_cache_copy: entry `to` = entry `from` for every pair, in each of n_pools pools
 *   (HOST array of DEVICE pointers, 16-byte aligned) of num_entries entries of
 *   entry_bytes (a multiple of 16). pairs: DEVICE int32 [n, 2]; those with a number
 *   outside the pool are skipped; count: DEVICE, only the first *count pairs (NULL:
 *   all n). No `to` may be another pair's `from` or `to`. Also copies entries of
 *   a KDA state pool or convolution-state pool, which a forked sequence needs of
 *   its own.
 * kda_cache_append: writes rows k, v (io dtype, [.., Hkv, D], ldk / ldv elements from
 *   one token to the next) to positions start[b], start[b] + 1, ... (DEVICE int32 [N])
 *   of sequences b = 0 .. N - 1 (table rows), whose pages must be there:
 *     cu_seqlens given (DEVICE int32 [N + 1]): packed rows, T = their total;
 *     else [N, T] rows, of sequence b the first count[b] (DEVICE int32 [N], NULL: T)
 *     in the order of index (DEVICE int32 [N, T], NULL: 0, 1, ..): the accepted
 *     tokens of a draft.
 *   Rows without a valid page are skipped and flagged (workspace may be NULL: then
 *   not flagged). Positions must be distinct.
 */
size_t kda_cache_workspace_size(int32_t num_pages, int32_t rows);
int kda_cache_alloc(int32_t *block_table, int64_t table_ld, int32_t rows, int32_t table_cols,
                    const int32_t *want, int32_t *refs, int32_t num_pages, int32_t page_size,
                    void *workspace, size_t workspace_bytes, void *stream);
int kda_cache_fork(int32_t *block_table, int64_t table_ld, int32_t rows, int32_t table_cols,
                   int32_t *seq_lens, int32_t *refs, int32_t num_pages, int32_t page_size,
                   const int32_t *src, const int32_t *dst, int32_t n, int32_t *copies,
                   void *workspace, size_t workspace_bytes, void *stream);
int kda_cache_free(int32_t *block_table, int64_t table_ld, int32_t rows, int32_t table_cols,
                   int32_t *seq_lens, int32_t *refs, int32_t num_pages, const int32_t *which,
                   int32_t n, void *workspace, size_t workspace_bytes, void *stream);
int kda_cache_compact(int32_t *block_table, int64_t table_ld, int32_t rows, int32_t table_cols,
                      int32_t *refs, int32_t num_pages, int32_t *copies, int32_t *count,
                      void *workspace, size_t workspace_bytes, void *stream);
int kda_cache_copy(void *const *pools, int32_t n_pools, int64_t entry_bytes, int32_t num_entries,
                   const int32_t *pairs, int32_t n, const int32_t *count, void *stream);
int kda_cache_append(const void *k, const void *v, int64_t ldk, int64_t ldv,
                     const int32_t *cu_seqlens, int32_t N, int32_t T, const int32_t *index,
                     const int32_t *count, const int32_t *start, const int32_t *block_table,
                     int64_t table_ld, int32_t table_cols, int32_t num_pages, int32_t page_size,
                     int32_t Hkv, int32_t D, int32_t io, void *k_pages, void *v_pages,
                     void *workspace, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H */
