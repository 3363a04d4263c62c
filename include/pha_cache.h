/*
 * pha_cache.h -- C ABI of libpha, serving side: a paged cache of keys and values, attention of new
 * tokens over it, and the management of its pages. Conventions are those of pha.h (device pointers
 * owned by the caller, asynchronous on `stream`, no allocation, argument errors before any launch;
 * `stream` belongs to the calling thread's current device).
 *
 * The cache. One layer's keys are k_pages[n_pages][page_size][n_kv_heads][head_dim], its values
 * v_pages likewise; page_size is a power of two. page_table[.][max_pages] (int32) has a row per
 * sequence: token p of sequence b lies in page page_table[b][p / page_size], row p % page_size.
 * A sequence without tokens (length 0) holds no pages, and its row may hold anything. In the row of
 * one with tokens the entries behind its last page are -1, as pha_cache_reserve, _fork and _free leave
 * them: pha_cache_fork and _free go by the whole row and take every entry that names a page for one
 * that the sequence holds. (What no token lies in makes no difference to the other calls.) On the paired
 * path (pha.h) a page's bytes are read as [2 * page_size][n_kv_heads / 2][head_dim], so the same cache
 * serves it.
 * The calls that manage pages take all layers at once: k_cache[n_layers][n_pages][page_size]
 * [n_kv_heads][head_dim], v_cache likewise, and one page_table, kv_lens and page_refs for all of
 * them. page_refs[n_pages] (int32) counts the table entries that hold a page; 0 means free.
 *
 * Status words. `status` (int32, device, may be NULL) is raised to the largest code that the call
 * meets and never lowered: zero it once, read it when convenient. Codes: 1 = lengths or indexes out
 * of range (or the same sequence twice in a list), 3 = a kernel wait ran out, 4 = a page table
 * entry that is needed is no page, 5 = not enough free pages. pha_cache_fork, _reserve, _free and
 * _compact also leave the code of the call itself (0 = fine) and a count in the first bytes of
 * their workspace, where pha_attn_status reads them.
 */
#ifndef PHA_CACHE_H
#define PHA_CACHE_H

#include "pha.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * pha_attn_paged_workspace_bytes -- device workspace of pha_attn_paged_fwd with the same arguments
 *   (work list, partial results of split key ranges). 0 for invalid arguments. The number of ranges
 *   follows the shape, so the size does not grow with every argument: a workspace kept for varying
 *   steps has the largest size among them.
 */
size_t pha_attn_paged_workspace_bytes(int batch, int max_q, int max_kv, int total_q, int n_heads,
                                      int n_kv_heads, int head_dim, pha_dtype dtype, int window,
                                      int sinks, int paired);

/*
 * pha_attn_paged_fwd -- causal attention of each sequence's new tokens over its paged cache, which
 *   already holds the new tokens' own keys and values (pha_cache_append). Single tokens (decoding),
 *   chunks of a prompt and mixtures of both are one call.
 *   q: [total_q][n_heads][head_dim]; the new tokens of sequence b are rows [cu_seqlens[b],
 *      cu_seqlens[b+1]) (none is fine); o, lse likewise, lse float[total_q][n_heads] or NULL.
 *   kv_lens: int32[batch], tokens in the cache, the new ones included: new token i of b stands at
 *      position p = kv_lens[b] - (number of new tokens of b) + i.
 *   Query position p sees key position j iff j <= p and (window <= 0, or p - j < window, or
 *   j < sinks). window and sinks count key slots (on the paired path positions, lengths and pages
 *   double and heads halve, as in pha_attn_fwd). Pages no query sees are not read: their table
 *   entries may be -1 (pha_cache_trim). Keys and values of the positions that some query of the call
 *   sees must be finite. Everything else in the pool may hold anything: rows behind a sequence's last
 *   token, in its last page too, and rows between the sinks and its first query's window.
 *   max_q, max_kv: bounds of the new tokens and of kv_lens over the batch.
 *   Result: o = sum_j w_j v_j, w the softmax of scale * q.k_j over the visible keys; lse its
 *   logarithm of the sum of exponentials. scale <= 0 selects 1/sqrt(head_dim).
 *   bf16 with head_dim 64 or 128 (tensor cores, float32 accumulation; weights rounded to bf16 for
 *   the second product); f32 with head_dim 1 .. 128 (CUDA cores).
 *   Rows of q behind cu_seqlens[batch] are not touched. A sequence whose lengths are out of range
 *   (kv_lens < new tokens, beyond max_kv or max_pages * page_size, more than max_q new tokens, rows
 *   outside q) raises status 1 and its rows are not written; if cu_seqlens decreases anywhere, which
 *   rows are written is unspecified.
 *   A needed entry that is no page raises status 4; the rows that see it are then unspecified.
 *   Errors: PHA_ERR_INVALID (NULL or misaligned pointers, sizes, head counts as in pha_attn_fwd,
 *   page_size no power of two, n_pages * page_size * n_kv_heads or total_q * n_heads beyond
 *   2^31 - 1 rows, sinks < 0),
 *   PHA_ERR_UNSUPPORTED (type / head_dim), PHA_ERR_WORKSPACE.
 */
pha_status pha_attn_paged_fwd(const void* q, const void* k_pages, const void* v_pages,
                              const int32_t* page_table, int max_pages, int n_pages, int page_size,
                              const int32_t* cu_seqlens, const int32_t* kv_lens, int batch,
                              int max_q, int max_kv, int total_q, int n_heads, int n_kv_heads,
                              int head_dim, pha_dtype dtype, int window, int sinks, int paired,
                              float scale, void* o, float* lse, void* workspace,
                              size_t workspace_bytes, int32_t* status, pha_stream_t stream);

/*
 * pha_test_attn_paged_fwd_stalled -- failure-detection test hook; not for production use.
 *   pha_attn_paged_fwd (same arguments, same checks) whose softmax warps first wait up to stall_us
 *   microseconds on a barrier that nothing signals: status 3, every role winds down, no row of o or
 *   lse is written. The GPU context and the workspace stay usable, as with
 *   pha_test_attn_fwd_stalled. stall_us: 1 .. 100000, else PHA_ERR_INVALID; f32 and calls of few rows
 *   a sequence (bf16, max_q times the heads of a group at most 16) have no waits: PHA_ERR_UNSUPPORTED.
 */
pha_status pha_test_attn_paged_fwd_stalled(const void* q, const void* k_pages, const void* v_pages,
                                           const int32_t* page_table, int max_pages, int n_pages,
                                           int page_size, const int32_t* cu_seqlens,
                                           const int32_t* kv_lens, int batch, int max_q, int max_kv,
                                           int total_q, int n_heads, int n_kv_heads, int head_dim,
                                           pha_dtype dtype, int window, int sinks, int paired,
                                           float scale, void* o, float* lse, void* workspace,
                                           size_t workspace_bytes, int32_t* status, int stall_us,
                                           pha_stream_t stream);

/*
 * pha_cache_append -- writes the new tokens' keys and values (rotated already: pha_rope) to their
 *   places in one layer's pages. k, v: [total][n_kv_heads][head_dim]; cu_seqlens, kv_lens (new
 *   tokens included), page_table as pha_attn_paged_fwd. Any type: element_bytes is 1, 2 or 4 (1 for
 *   caches that other code reads: pha_attn_paged_fwd takes bf16 and f32), and n_kv_heads * head_dim *
 *   element_bytes a multiple of 16.
 *   A token whose place is out of range (status 1) or whose entry is no page (status 4) is left out.
 *   No two tokens may have one place (pages shared by sequences are not written: pha_cache_reserve
 *   copies the one a sequence grows into).
 */
pha_status pha_cache_append(const void* k, const void* v, void* k_pages, void* v_pages,
                            const int32_t* page_table, int max_pages, int n_pages, int page_size,
                            const int32_t* cu_seqlens, const int32_t* kv_lens, int batch, int total,
                            int n_kv_heads, int head_dim, int element_bytes, int32_t* status,
                            pha_stream_t stream);

/* pha_cache_workspace_bytes -- device workspace of the four calls below. 0 for invalid arguments. */
size_t pha_cache_workspace_bytes(int n_pages, int n_seqs);

/*
 * pha_cache_fork -- sequence dst[i] becomes a second holder of src[i]'s pages (nothing is copied):
 *   its table row and length are src[i]'s and each page held counts one more in page_refs.
 *   src, dst: int32[n] on the device; every dst[i] must be an empty sequence (length 0), named once,
 *   and no src. One source may be forked many times in one call. Count: pages shared.
 *   Anything out of range: status 1, nothing changed.
 */
pha_status pha_cache_fork(int32_t* page_table, int max_pages, int32_t* kv_lens, int n_seqs,
                          int32_t* page_refs, int n_pages, const int32_t* src, const int32_t* dst,
                          int n, void* workspace, size_t workspace_bytes, int32_t* status,
                          pha_stream_t stream);

/*
 * pha_cache_reserve -- room for new_tokens[i] more tokens of sequence seqs[i] (each named once):
 *   kv_lens grows by them and the table gets the pages they need, lowest free page first, in the
 *   order of the list (an empty sequence's row becomes -1 behind them). A sequence that grows into a
 *   last page that it shares (page_refs > 1 before the call) gets a page of its own with the shared
 *   one's contents, in all layers, first.
 *   page_bytes: bytes of one page of one layer and of K or V alone (page_size * n_kv_heads * head_dim
 *   * element size), a multiple of 16.
 *   Too few free pages: status 5; out of range, or longer than max_pages pages or 2^31 - 1 tokens:
 *   status 1; a last page that is none: status 4. Nothing is changed then. Count: pages taken.
 */
pha_status pha_cache_reserve(int32_t* page_table, int max_pages, int32_t* kv_lens, int n_seqs,
                             int32_t* page_refs, int n_pages, int page_size, const int32_t* seqs,
                             const int32_t* new_tokens, int n, void* k_cache, void* v_cache,
                             int n_layers, size_t page_bytes, void* workspace,
                             size_t workspace_bytes, int32_t* status, pha_stream_t stream);

/*
 * pha_cache_free -- sequences seqs[i] (each named once) let go of their pages: page_refs goes down,
 *   table rows become -1, lengths 0. A page whose count reaches 0 is free. Count: entries let go.
 *   Out of range: status 1, nothing changed.
 */
pha_status pha_cache_free(int32_t* page_table, int max_pages, int32_t* kv_lens, int n_seqs,
                          int32_t* page_refs, int n_pages, const int32_t* seqs, int n,
                          void* workspace, size_t workspace_bytes, int32_t* status,
                          pha_stream_t stream);

/*
 * pha_cache_trim -- every sequence lets go of the pages that no later token sees with this window
 *   (> 0) and these sinks: page e goes when e * page_size >= sinks and (e + 1) * page_size <=
 *   kv_lens - window + 1 (in slots; paired doubles the page and the length). Table entries become
 *   -1; lengths stay.
 */
pha_status pha_cache_trim(int32_t* page_table, int max_pages, const int32_t* kv_lens, int n_seqs,
                          int32_t* page_refs, int n_pages, int page_size, int window, int sinks,
                          int paired, int32_t* status, pha_stream_t stream);

/*
 * pha_cache_compact -- moves the pages in use together: with n_live pages in use, those at n_live
 *   and behind move, in order, into the free pages before it (all layers, K and V), and page_table
 *   and page_refs follow. Pages [0, n_live) are then in use and the rest is free. Table entries of
 *   value -1 stay. Count: pages moved.
 */
pha_status pha_cache_compact(int32_t* page_table, int max_pages, int n_seqs, int32_t* page_refs,
                             int n_pages, void* k_cache, void* v_cache, int n_layers,
                             size_t page_bytes, void* workspace, size_t workspace_bytes,
                             int32_t* status, pha_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PHA_CACHE_H */
