/* Entry points of the TEST library only (libmla_b200_test.so, built from the
 * same sources with MLA_TEST_ENTRY_POINTS defined, plus the SIMT kernel).
 * The product library libmla_b200.so does not export them. */
#pragma once

#include "../../include/mla.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The decode of mla_decode_fwd computed by a plain SIMT kernel (fp32 FMA,
 * no tensor cores) over the same schedule and workspace: a second,
 * independently written device implementation for the parity tests.
 * Arguments, layouts and errors as for mla_decode_fwd. */
int mla_decode_fwd_simt(const mla_shape_t* shape, const void* q, const void* kv_cache,
                        const float* kv_scale, const int32_t* block_table,
                        const int32_t* seqlens, float softmax_scale, const void* sched,
                        void* workspace, size_t workspace_bytes, void* out, float* lse,
                        void* stream);

/* mla_decode_fwd with the decode kernel's test hook set: one of its bounded
 * waits waits on a barrier that nothing arrives on, runs out after about
 * 2 s, and the kernel's abort path runs (status bit, both CTAs stop, copies
 * and MMAs drained, tensor memory freed).  mla_get_device_status then
 * reports MLA_ERR_TIMEOUT; the outputs are not valid.  Faults nothing. */
int mla_test_decode_stalled(const mla_shape_t* shape, const void* q, const void* kv_cache,
                            const float* kv_scale, const int32_t* block_table,
                            const int32_t* seqlens, float softmax_scale, const void* sched,
                            void* workspace, size_t workspace_bytes, void* out, float* lse,
                            void* stream);

/* mla_attn_weights_fwd with its kernel's test hook set: the MMA issuers wait
 * on a barrier that nothing arrives on, which runs out after about 2 s and
 * runs the abort path.  mla_attn_weights_get_device_status then reports
 * MLA_ERR_TIMEOUT; the weights are not valid.  Faults nothing. */
int mla_test_attn_weights_stalled(const mla_shape_t* shape, const void* q, const void* kv_cache, const float* kv_scale,
                                  const int32_t* block_table, const int32_t* seqlens, const float* lse,
                                  float softmax_scale, float decay, float* weights, void* workspace,
                                  size_t workspace_bytes, void* stream);

/* The host copy of the tree decode's scheduler (mla_plan_schedule_host for
 * mla_tree_decode_fwd's schedule, which lies at the head of its workspace):
 * seqlens, draft_lens (or NULL) and sched are HOST pointers. */
int mla_test_plan_tree_schedule_host(const mla_shape_t* shape, const int32_t* seqlens, const int32_t* draft_lens, int num_sms,
                                     void* sched, size_t sched_bytes);

/* mla_cache_compact with its kernel's test hook set: the groups whose rows
 * go where rows of a request's first group lay are never told that those
 * have been read; their waits run out after about 2 s each.
 * mla_compact_get_device_status then reports MLA_ERR_TIMEOUT and the rows of
 * those requests are not valid.  Faults nothing. */
int mla_test_compact_stalled(const mla_shape_t* shape, void* kv_cache, float* kv_scale, const int32_t* block_table,
                             const int32_t* src, const int32_t* src_lens, const int32_t* base, int32_t max_rows,
                             float* weights, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
