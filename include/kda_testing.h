/*
 * kda_testing.h -- entry points of libkda.so that exist only for tests of its
 * failure detection. Production code never calls them; nothing in kda.h
 * reaches them, and no environment variable switches them on.
 */
#ifndef KDA_TESTING_H
#define KDA_TESTING_H

#include <stddef.h>
#include <stdint.h>

#include "kda.h"  /* kda_prefill_plan_info */

#ifdef __cplusplus
extern "C" {
#endif

/*
 * kda_prefill (bf16 I/O only, arguments as there) with its recurrence chains
 * launched WITHOUT the chunk-preparation producers of the fused schedule and
 * with every wait of a chain bounded by wait_ms milliseconds (1..10000). No
 * ready flag is ever set, so each chain gives up after wait_ms, records
 * KDA_ERR_TIMEOUT in the workspace status word (read it with
 * kda_workspace_status) and returns; the outputs are garbage. It shows that a
 * missing producer ends in an error status and a usable context, never in a
 * hang. Needs fewer chains (N * H) than SMs. Returns KDA_OK once enqueued,
 * KDA_ERR_UNSUPPORTED for fp32 I/O, KDA_ERR_INVALID_ARG for a bad wait_ms or
 * invalid arguments, KDA_ERR_CUDA if the launch fails (e.g. too many chains).
 * The pages have no counterpart to this entry point.
 */
int kda_testing_prefill_chain_timeout(const void *q, const void *k, const void *v,
                                      const float *g, const void *beta, float scale,
                                      const float *init_state, const int32_t *cu_seqlens,
                                      int32_t N, int32_t T, int32_t H, int32_t D, int32_t chunk,
                                      int32_t io, void *out, float *final_state, void *workspace,
                                      size_t workspace_bytes, int32_t wait_ms, void *stream);

/*
 * The workspace-plan selection of the bf16 prefill (the host logic behind
 * kda_prefill_plan) for given device properties instead of the current
 * device's, so that it can be checked without a GPU: sm_count SMs,
 * cooperative != 0 if cooperative launches are supported, schedule_override
 * -1 (automatic), KDA_SCHEDULE_SPLIT or KDA_SCHEDULE_FUSED. kind 0: the plan
 * that a workspace of workspace_bytes gets; 1: the fastest plan; 2: the ring
 * plan with the modelled best group; 3: the smallest accepted plan (kinds 1-3
 * ignore workspace_bytes). Sizes as in kda_prefill_workspace_size (D = 128,
 * chunk 64). Writes *plan and returns KDA_OK; KDA_ERR_INVALID_ARG when the
 * arguments are invalid or no plan fits. Launches nothing, needs no device.
 */
int kda_testing_prefill_plan(int32_t N, int32_t T, int32_t H, int32_t varlen, int32_t sm_count,
                             int32_t cooperative, int32_t schedule_override, int32_t kind,
                             size_t workspace_bytes, kda_prefill_plan_info *plan);

/*
 * kda_attn_prefill and kda_attn_decode (bf16 I/O only, arguments as there) in which, in
 * every CTA, one warp gives up at one of its waits, as if its limit of 20
 * milliseconds (two seconds in production) had run out: warp 0..7 of the softmax,
 * 8 products, 9 copies, 10 scheduler, 11 zeros past a sequence's end; `at` counts that
 * warp's waits from 0. What the others wait for then never comes, so every role gives up
 * within its limits, the call records KDA_ERR_TIMEOUT in the workspace's status word
 * and returns; the outputs are garbage. (A warp that has fewer waits than that never gives
 * up: the call is then an ordinary one.) It shows that a role that stops ends in an
 * error status and a usable context, never in a hang. KDA_ERR_INVALID_ARG for another io,
 * warp or at.
 */
int kda_testing_attn_prefill_timeout(const void *q, const void *k, const void *v, int64_t ldq,
                                     int64_t ldk, int64_t ldv, float scale,
                                     const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k,
                                     int32_t N, int32_t Tq, int32_t Tk, int32_t Hq, int32_t Hkv,
                                     int32_t D, int32_t io, void *out, float *lse, void *workspace,
                                     size_t workspace_bytes, int32_t warp, int32_t at,
                                     void *stream);
int kda_testing_attn_decode_timeout(const void *q, int64_t ldq, const void *k_new,
                                    const void *v_new, int64_t ldk, int64_t ldv,
                                    const void *k_pages, const void *v_pages, int32_t num_pages,
                                    int32_t page_size, const int32_t *block_table,
                                    int64_t table_ld, int32_t table_cols, const int32_t *seq_lens,
                                    const uint64_t *tree_mask, float scale, int32_t B, int32_t T,
                                    int32_t Hq, int32_t Hkv, int32_t D, int32_t io, void *out,
                                    float *lse, void *workspace, size_t workspace_bytes,
                                    int32_t warp, int32_t at, void *stream);

/* kda_attn_prefill_window and kda_attn_decode_window likewise. */
int kda_testing_attn_prefill_window_timeout(const void *q, const void *k, const void *v,
                                            int64_t ldq, int64_t ldk, int64_t ldv, float scale,
                                            int32_t window, int32_t sinks,
                                            const int32_t *cu_seqlens_q,
                                            const int32_t *cu_seqlens_k, int32_t N, int32_t Tq,
                                            int32_t Tk, int32_t Hq, int32_t Hkv, int32_t D,
                                            int32_t io, void *out, float *lse, void *workspace,
                                            size_t workspace_bytes, int32_t warp, int32_t at,
                                            void *stream);
int kda_testing_attn_decode_window_timeout(const void *q, int64_t ldq, const void *k_new,
                                           const void *v_new, int64_t ldk, int64_t ldv,
                                           const void *k_pages, const void *v_pages,
                                           int32_t num_pages, int32_t page_size,
                                           const int32_t *block_table, int64_t table_ld,
                                           int32_t table_cols, const int32_t *seq_lens,
                                           const uint64_t *tree_mask, float scale, int32_t window,
                                           int32_t sinks, int32_t B, int32_t T, int32_t Hq,
                                           int32_t Hkv, int32_t D, int32_t io, void *out,
                                           float *lse, void *workspace, size_t workspace_bytes,
                                           int32_t warp, int32_t at, void *stream);

/*
 * kda_attn_weights likewise (bf16 I/O only, arguments as there): warp 0..15 of the
 * exponentials, 16 products, 17 copies of keys, 18..21 rows, of which 18 walks the parts. The weights
 * are garbage afterwards.
 */
int kda_testing_attn_weights_timeout(const void *q, int64_t ldq, const void *k_pages,
                                     int32_t num_pages, int32_t page_size,
                                     const int32_t *block_table, int64_t table_ld,
                                     int32_t table_cols, const int32_t *seq_lens, const float *lse,
                                     const int32_t *index, const int32_t *count, float scale,
                                     int32_t B, int32_t T, int32_t Hq, int32_t Hkv, int32_t D,
                                     int32_t io, float *weights, int32_t cap, void *workspace,
                                     int32_t warp, int32_t at, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_TESTING_H */
