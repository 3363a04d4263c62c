/*
 * pha_sinks.h -- C ABI of libpha: causal varlen attention with a sliding window and visible first
 * slots (sinks), forward and backward. Conventions, layouts and the paired view are those of pha.h.
 *
 * Query slot i of the document [a, b) sees key slot j iff a <= j <= i and (i - j < window or
 * j - a < sinks). window and sinks count key slots (neither is doubled on the paired path);
 * window <= 0 means no window (the sinks then change nothing).
 */
#ifndef PHA_SINKS_H
#define PHA_SINKS_H

#include "pha.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Device workspace of pha_attn_sinks_fwd / pha_attn_sinks_bwd with the same arguments. 0 for
 * invalid ones. */
size_t pha_attn_sinks_workspace_bytes(int batch, int max_len, int n_heads, int n_kv_heads,
                                      int head_dim, int window, int sinks, int paired);
size_t pha_attn_sinks_bwd_workspace_bytes(int batch, int max_len, int total_tokens, int n_heads,
                                          int n_kv_heads, int head_dim, int window, int sinks,
                                          int paired);

/*
 * pha_attn_sinks_fwd -- o and lse as pha_attn_fwd defines them, over the keys above. Arguments,
 *   supported types (bf16 with head_dim 64 / 128; f32 with head_dim 1 .. 128), device status
 *   (pha_attn_status(workspace)) and errors as pha_attn_fwd with causal = 1, and:
 *   sinks: 0 <= sinks, else PHA_ERR_INVALID; more than 128: PHA_ERR_UNSUPPORTED.
 *   total_tokens * n_heads beyond 2^31 - 1 rows, batch * min(max_len, 2^29) beyond 2^48:
 *   PHA_ERR_INVALID.
 *   workspace: pha_attn_sinks_workspace_bytes(...) bytes, needed for f32 too. Rows outside every
 *   document are not written. k and v rows inside the documents must be finite.
 */
pha_status pha_attn_sinks_fwd(const void* q, const void* k, const void* v,
                              const int32_t* cu_seqlens, int batch, int max_len, int total_tokens,
                              int n_heads, int n_kv_heads, int head_dim, pha_dtype dtype,
                              int window, int sinks, int paired, float scale, void* o, float* lse,
                              void* workspace, size_t workspace_bytes, pha_stream_t stream);

/*
 * pha_attn_sinks_bwd -- dq, dk, dv of pha_attn_sinks_fwd for the upstream gradient dout; arguments,
 *   arithmetic and errors as pha_attn_bwd with the mask above. o, lse: the forward's outputs. Rows
 *   outside every document get zeros. No atomics: the same inputs give the same bits. Malformed
 *   cu_seqlens: status 1 (pha_attn_status(workspace)); no gradient is computed, rows outside
 *   [cu_seqlens[0], cu_seqlens[batch]) may get their zeros all the same.
 */
pha_status pha_attn_sinks_bwd(const void* q, const void* k, const void* v, const void* o,
                              const float* lse, const void* dout, const int32_t* cu_seqlens,
                              int batch, int max_len, int total_tokens, int n_heads,
                              int n_kv_heads, int head_dim, pha_dtype dtype, int window, int sinks,
                              int paired, float scale, void* dq, void* dk, void* dv,
                              void* workspace, size_t workspace_bytes, pha_stream_t stream);

/*
 * pha_test_attn_sinks_fwd_stalled, pha_test_attn_sinks_bwd_stalled -- failure-detection test hooks; not
 *   for production use. The call of the same name without test_ and _stalled (same arguments, same
 *   checks), whose softmax (elementwise) warps first wait up to stall_us microseconds on a barrier
 *   that nothing signals: device status 3, every role winds down, and no row of o, lse, dq, dk or dv
 *   inside a document is written. The GPU context and the workspace stay usable, as with
 *   pha_test_attn_fwd_stalled. stall_us: 1 .. 100000, else PHA_ERR_INVALID; PHA_F32 has no waits:
 *   PHA_ERR_UNSUPPORTED.
 */
pha_status pha_test_attn_sinks_fwd_stalled(const void* q, const void* k, const void* v,
                                           const int32_t* cu_seqlens, int batch, int max_len,
                                           int total_tokens, int n_heads, int n_kv_heads,
                                           int head_dim, pha_dtype dtype, int window, int sinks,
                                           int paired, float scale, void* o, float* lse,
                                           void* workspace, size_t workspace_bytes, int stall_us,
                                           pha_stream_t stream);
pha_status pha_test_attn_sinks_bwd_stalled(const void* q, const void* k, const void* v,
                                           const void* o, const float* lse, const void* dout,
                                           const int32_t* cu_seqlens, int batch, int max_len,
                                           int total_tokens, int n_heads, int n_kv_heads,
                                           int head_dim, pha_dtype dtype, int window, int sinks,
                                           int paired, float scale, void* dq, void* dk, void* dv,
                                           void* workspace, size_t workspace_bytes, int stall_us,
                                           pha_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PHA_SINKS_H */
