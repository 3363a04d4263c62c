// cache.cuh -- arguments of the page kernels (cache.cu) as pha_cache.cu passes them.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace pha {

struct AppendArgs {
    const uint4* k;
    const uint4* v;
    uint4* k_pages;
    uint4* v_pages;
    const int32_t* table;
    const int32_t* cu;
    const int32_t* kv_lens;
    int32_t* status;
    int max_pages, n_pages, page_shift, batch, total;
    int row_units;  // 16-byte units of one token's keys
};

// First bytes of the workspace; n_items and status stand where pha_attn_status reads them.
struct CacheHeader {
    int n_items;   // the call's count
    int status;
    int n_copies;  // entries of copy_src / copy_dst for the copy kernel
    int n_live;    // compact: pages in use
};

struct CacheArgs {
    int32_t* table;
    int32_t* lens;
    int32_t* refs;
    int32_t* status;
    int max_pages, n_seqs, n_pages;
    CacheHeader* hdr;
    int32_t* marks;     // [n_seqs] which sequences the call's list names
    int32_t* need;      // [n_seqs] reserve: pages list entry i takes
    int32_t* first;     // [n_seqs] reserve: ... from this place of `pages` on
    int32_t* copy_src;  // [max(n_seqs, n_pages)] pages to copy (-1: none)
    int32_t* copy_dst;
    int32_t* pages;     // [n_pages] reserve: pages handed out; compact: a moved page's new place
};

cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t stream);
cudaError_t launch_cache_fork(const CacheArgs& c, const int32_t* src, const int32_t* dst, int n,
                              cudaStream_t stream);
cudaError_t launch_cache_free(const CacheArgs& c, const int32_t* seqs, int n, cudaStream_t stream);
cudaError_t launch_cache_reserve(const CacheArgs& c, const int32_t* seqs, const int32_t* new_tokens,
                                 int n, int page_shift, void* k_cache, void* v_cache, int n_layers,
                                 size_t page_bytes, cudaStream_t stream);
cudaError_t launch_cache_trim(const CacheArgs& c, int page_size, int window, int sinks, int mult,
                              cudaStream_t stream);
cudaError_t launch_cache_compact(const CacheArgs& c, void* k_cache, void* v_cache, int n_layers,
                                 size_t page_bytes, cudaStream_t stream);

}  // namespace pha
