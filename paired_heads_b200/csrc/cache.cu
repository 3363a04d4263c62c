// cache.cu -- the pages of the key / value cache: writing new tokens to them, and the integer work
// of forking, reserving, freeing, trimming and compacting (include/pha_cache.h).
//
// What bounds these: pha_cache_append and the page copies of reserve / compact move bytes (read
// once, written once); everything else is a few kilobytes of table and counts, so its time is
// launches and dependent loads. The integer part of a call is one CTA that checks every argument
// found in device memory before it changes anything -- "nothing changed" on an error needs all
// checks to precede all writes -- and hands the copies to a second, grid-wide kernel through a list
// in the workspace. Page numbers are handed out by scans in index order, never by the order in
// which atomics arrive, so the same state and call give the same tables. Measured: append 99 us for 596 MB
// (6.0 TB/s); the copies of a compaction 156 us for 863 MB (5.5 TB/s) behind 8 us of list; fork, reserve and
// free of 64 sequences 6, 9 and 4 us.
#include <cuda_runtime.h>
#include <stdint.h>

#include "cache.cuh"
#include "kernels.cuh"
#include "scan.cuh"

namespace pha {

namespace {

constexpr int kThreads = 1024;        // the one-CTA kernels
constexpr int kPerThread = 8;         // page counts a thread looks at per chunk of a page scan
constexpr int kCopyThreads = 256;
constexpr int kCopyUnits = 4;         // 16-byte units a thread has in flight

__device__ __forceinline__ void raise(int32_t* status, int code) {
    if (status && code != DEV_OK) atomicMax(status, code);
}

// ------------------------------------------------------------------------------------- append

// Sequence of new token t: the last b with cu[b] <= t (-1: before the first).
__device__ __forceinline__ int seq_of_token(const int32_t* __restrict__ cu, int batch, int t) {
    int lo = -1, hi = batch;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(cu + mid) <= t) lo = mid; else hi = mid;
    }
    return lo;
}

// Row of the pool (page * page_size + row in the page) that token t goes to; -1: nowhere.
__device__ __forceinline__ int64_t place_of_token(const AppendArgs& a, int t, int& code) {
    const int b = seq_of_token(a.cu, a.batch, t);
    if (b < 0) return -1;
    const int c0 = __ldg(a.cu + b), c1 = __ldg(a.cu + b + 1);
    if (t >= c1) return -1;  // behind the last sequence
    const int64_t pos = static_cast<int64_t>(__ldg(a.kv_lens + b)) - c1 + t;
    if (c0 < 0 || c1 > a.total || pos < 0 || pos + c0 < t || (pos >> a.page_shift) >= a.max_pages) {
        code = DEV_BAD_SEQLENS;
        return -1;
    }
    const int page = __ldg(a.table + static_cast<int64_t>(b) * a.max_pages + (pos >> a.page_shift));
    if (page < 0 || page >= a.n_pages) {
        code = DEV_BAD_PAGE;
        return -1;
    }
    return (static_cast<int64_t>(page) << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
}

// Thread = 16-byte units x of K and of V, flat over (token, unit of its row).
__global__ void __launch_bounds__(kCopyThreads) append_kernel(AppendArgs a) {
    const int64_t n = static_cast<int64_t>(a.total) * a.row_units;
    for (int64_t x = static_cast<int64_t>(blockIdx.x) * kCopyThreads + threadIdx.x; x < n;
         x += static_cast<int64_t>(gridDim.x) * kCopyThreads) {
        const int t = static_cast<int>(x / a.row_units), u = static_cast<int>(x % a.row_units);
        const uint4 k = __ldg(a.k + x), v = __ldg(a.v + x);
        int code = DEV_OK;
        const int64_t row = place_of_token(a, t, code);
        if (u == 0) raise(a.status, code);
        if (row < 0) continue;
        a.k_pages[row * a.row_units + u] = k;
        a.v_pages[row * a.row_units + u] = v;
    }
}

// --------------------------------------------------------------------------- one-CTA bookkeeping

// The result of the call in the workspace header and the status word; uniform over the CTA.
__device__ __forceinline__ void finish(const CacheArgs& c, int code, int count) {
    if (threadIdx.x == 0) {
        c.hdr->n_items = code == DEV_OK ? count : 0;
        c.hdr->status = code;
        raise(c.status, code);
    }
}

// The largest code over the CTA (every thread calls it and gets it).
__device__ __forceinline__ int cta_code(int code, int* shared_code) {
    if (threadIdx.x == 0) *shared_code = DEV_OK;
    __syncthreads();
    if (code != DEV_OK) atomicMax(shared_code, code);
    __syncthreads();
    const int worst = *shared_code;
    __syncthreads();
    return worst;
}

__device__ __forceinline__ bool is_seq(const CacheArgs& c, int s) { return s >= 0 && s < c.n_seqs; }

// Whether list[0 .. n) names sequences in range, each once; src[0 .. n) (may be NULL) sequences in
// range. Afterwards c.marks of all of them is 1 for those in the list and 0 for the others.
__device__ int check_list(const CacheArgs& c, const int32_t* list, const int32_t* src, int n,
                          int* shared_code) {
    int code = DEV_OK;
    for (int i = threadIdx.x; i < n; i += kThreads) {
        if (is_seq(c, list[i]) && (!src || is_seq(c, src[i]))) {
            c.marks[list[i]] = 0;
            if (src) c.marks[src[i]] = 0;
        } else {
            code = DEV_BAD_SEQLENS;
        }
    }
    code = cta_code(code, shared_code);
    if (code != DEV_OK) return code;
    for (int i = threadIdx.x; i < n; i += kThreads)
        if (atomicAdd(&c.marks[list[i]], 1) != 0) code = DEV_BAD_SEQLENS;
    return cta_code(code, shared_code);
}

// Warp per sequence of the list, lanes over its table row. fork: dst takes over src's row and each
// page gains a holder; otherwise (free) the sequence's pages lose one. A sequence without tokens holds no
// pages, whatever its row says. Returns the entries handled.
template <bool FORK>
__device__ int share_or_drop(const CacheArgs& c, const int32_t* src, const int32_t* list, int n,
                             int first_warp, int n_warps) {
    const int lane = threadIdx.x & 31;
    int count = 0;
    for (int i = first_warp; i < n; i += n_warps) {
        int32_t* to = c.table + static_cast<int64_t>(list[i]) * c.max_pages;
        const int32_t* from = FORK ? c.table + static_cast<int64_t>(src[i]) * c.max_pages : to;
        const int len = c.lens[FORK ? src[i] : list[i]];
        __syncwarp();  // (every lane has it before lane 0 writes the new one)
        for (int j = lane; j < c.max_pages; j += 32) {
            const int page = len > 0 ? from[j] : -1;
            if (page >= 0 && page < c.n_pages) {
                atomicAdd(&c.refs[page], FORK ? 1 : -1);
                ++count;
            }
            to[j] = FORK ? page : -1;
        }
        if (lane == 0) c.lens[list[i]] = FORK ? len : 0;
    }
    return count;
}

template <bool FORK>
__global__ void __launch_bounds__(kThreads) share_kernel(CacheArgs c, const int32_t* src,
                                                         const int32_t* list, int n) {
    __shared__ int shared_code;
    __shared__ int sums[kThreads / 32];
    int code = check_list(c, list, src, n, &shared_code);
    if (FORK && code == DEV_OK) {
        for (int i = threadIdx.x; i < n; i += kThreads)  // no source is a destination too
            if (c.lens[list[i]] != 0 || c.marks[src[i]] != 0) code = DEV_BAD_SEQLENS;
        code = cta_code(code, &shared_code);
    }
    if (code != DEV_OK) return finish(c, code, 0);
    const int mine = share_or_drop<FORK>(c, src, list, n, threadIdx.x >> 5, kThreads / 32);
    int total;
    cta_exclusive_scan<kThreads>(mine, sums, total);
    finish(c, DEV_OK, total);
}

// --------------------------------------------------------------------------------- page scans

// Walks the pages [begin, end) in chunks of kThreads * kPerThread, thread t of the CTA looking at
// kPerThread consecutive ones; emit(rank, page) for each page with wanted(refs[page]), rank counting
// them from `done`. Stops after `most` of them. Returns done + the number found (at most `most`
// beyond what was asked is counted, never emitted past it).
template <typename Wanted, typename Emit>
__device__ int scan_pages(const int32_t* refs, int begin, int end, int done, int most, int* sums,
                          Wanted wanted, Emit emit) {
    for (int64_t base = begin; base < end && done < most; base += kThreads * kPerThread) {
        const int64_t p0 = base + static_cast<int64_t>(threadIdx.x) * kPerThread;
        uint32_t bits = 0;
#pragma unroll
        for (int e = 0; e < kPerThread; ++e)
            if (p0 + e < end && wanted(refs[p0 + e])) bits |= 1u << e;
        int total;
        int rank = done + cta_exclusive_scan<kThreads>(__popc(bits), sums, total);
#pragma unroll
        for (int e = 0; e < kPerThread; ++e)
            if ((bits >> e) & 1u) {
                if (rank < most) emit(rank, static_cast<int>(p0 + e));
                ++rank;
            }
        done += total;
    }
    return done;
}

// -------------------------------------------------------------------------------------- reserve

__global__ void __launch_bounds__(kThreads) reserve_kernel(CacheArgs c, const int32_t* seqs,
                                                           const int32_t* new_tokens, int n,
                                                           int page_shift) {
    __shared__ int shared_code;
    __shared__ int sums[kThreads / 32];
    __shared__ int64_t needs[kThreads / 32];
    grid_dep_launch();  // the copy kernel may come up; it waits for this one's end
    const int page_size = 1 << page_shift;
    int code = check_list(c, seqs, nullptr, n, &shared_code);
    // what each sequence needs: its own copy of a shared last page, then pages for the rest
    int64_t total = 0;
    if (code == DEV_OK) {
        for (int base = 0; base < n; base += kThreads) {
            const int i = base + threadIdx.x;
            int64_t need = 0;
            if (i < n) {
                const int s = seqs[i];
                const int64_t len = c.lens[s], grow = new_tokens[i];
                const int64_t have = (len + page_size - 1) >> page_shift;
                const int64_t want = (len + grow + page_size - 1) >> page_shift;
                int shared_page = -1;
                if (len < 0 || grow < 0 || len + grow > INT32_MAX || want > c.max_pages) {
                    code = DEV_BAD_SEQLENS;
                } else if (grow > 0 && (len & (page_size - 1)) != 0) {
                    const int last = c.table[static_cast<int64_t>(s) * c.max_pages + have - 1];
                    if (last < 0 || last >= c.n_pages) code = DEV_BAD_PAGE;
                    else if (c.refs[last] > 1) shared_page = last;
                }
                if (code == DEV_OK) need = want - have + (shared_page >= 0 ? 1 : 0);
                c.copy_src[i] = shared_page;
                c.need[i] = static_cast<int>(need);
            }
            int64_t chunk;
            const int64_t before = cta_exclusive_scan<kThreads>(need, needs, chunk);
            if (i < n) c.first[i] = static_cast<int>(total + before);  // (read only if the pool has them all)
            total += chunk;
        }
        code = cta_code(code, &shared_code);
    }
    // the lowest free pages, as many as needed
    if (code == DEV_OK && total > 0) {
        int found = 0;
        if (total <= c.n_pages)
            found = scan_pages(c.refs, 0, c.n_pages, 0, static_cast<int>(total), sums,
                               [](int r) { return r == 0; }, [&](int rank, int page) { c.pages[rank] = page; });
        if (found < total) code = DEV_NO_PAGES;
        __syncthreads();  // the list is read by other threads next
    }
    if (code != DEV_OK) {
        if (threadIdx.x == 0) c.hdr->n_copies = 0;
        return finish(c, code, 0);
    }
    // hand them out: warp per sequence, lanes over its new pages
    const int lane = threadIdx.x & 31;
    for (int i = threadIdx.x >> 5; i < n; i += kThreads / 32) {
        const int s = seqs[i];
        const int64_t len = c.lens[s];
        const int old = c.copy_src[i], need = c.need[i];
        const int64_t at = ((len + page_size - 1) >> page_shift) - (old >= 0 ? 1 : 0);
        __syncwarp();  // (every lane has the length before lane 0 writes the new one)
        for (int j = lane; j < need; j += 32) {
            const int page = c.pages[c.first[i] + j];
            c.table[static_cast<int64_t>(s) * c.max_pages + at + j] = page;
            c.refs[page] = 1;
        }
        if (len == 0 && need > 0)  // the row may hold anything so far; fork and free go by all of it
            for (int64_t j = need + lane; j < c.max_pages; j += 32) c.table[static_cast<int64_t>(s) * c.max_pages + j] = -1;
        if (lane == 0) {
            c.copy_dst[i] = old >= 0 ? c.pages[c.first[i]] : -1;
            if (old >= 0) atomicSub(&c.refs[old], 1);
            c.lens[s] = static_cast<int>(len + new_tokens[i]);
        }
    }
    if (threadIdx.x == 0) c.hdr->n_copies = n;
    finish(c, DEV_OK, static_cast<int>(total));
}

// -------------------------------------------------------------------------------------- compact

__global__ void __launch_bounds__(kThreads) compact_kernel(CacheArgs c) {
    __shared__ int sums[kThreads / 32];
    grid_dep_launch();
    int mine = 0, live;
    for (int64_t p = threadIdx.x; p < c.n_pages; p += kThreads) mine += c.refs[p] > 0;
    cta_exclusive_scan<kThreads>(mine, sums, live);
    // pages at `live` and behind that nobody holds have no new place (a stale table entry stays)
    for (int64_t p = live + static_cast<int64_t>(threadIdx.x); p < c.n_pages; p += kThreads)
        if (c.refs[p] <= 0) c.pages[p] = -1;
    // as many live pages lie at `live` and behind as free ones lie before it
    const int moves = scan_pages(c.refs, live, c.n_pages, 0, c.n_pages, sums,
                                 [](int r) { return r > 0; },
                                 [&](int rank, int page) { c.copy_src[rank] = page; });
    scan_pages(c.refs, 0, live, 0, c.n_pages, sums, [](int r) { return r <= 0; },
               [&](int rank, int page) { c.copy_dst[rank] = page; });
    __syncthreads();
    for (int i = threadIdx.x; i < moves; i += kThreads) {
        const int from = c.copy_src[i], to = c.copy_dst[i];
        c.pages[from] = to;
        c.refs[to] = c.refs[from];
        c.refs[from] = 0;
    }
    if (threadIdx.x == 0) {
        c.hdr->n_copies = moves;
        c.hdr->n_live = live;
    }
    finish(c, DEV_OK, moves);
}

// ---------------------------------------------------------------------------------- page copies

// Copies pages copy_src[i] -> copy_dst[i] (entries with a negative one skipped) of every layer, K and
// V, in pieces of kPieceBytes; sources and destinations are different pages. retable: the table's
// entries at n_live and behind follow c.pages.
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(CacheArgs c, uint4* k_cache, uint4* v_cache,
                                                                  int n_layers, int64_t page_units,
                                                                  int retable) {
    grid_dep_wait();
    const int n = c.hdr->n_copies;
    constexpr int kUnits = kCopyThreads * kCopyUnits;
    const int64_t pieces = (page_units + kUnits - 1) / kUnits;
    const int64_t per_copy = pieces * n_layers * 2;
    for (int64_t w = blockIdx.x; w < n * per_copy; w += gridDim.x) {
        const int64_t i = w / per_copy;
        const int from = c.copy_src[i];
        if (from < 0) continue;
        const int to = c.copy_dst[i];
        int64_t r = w % per_copy;
        uint4* cache = (r & 1) ? v_cache : k_cache;
        r >>= 1;
        const int64_t layer = (r / pieces) * c.n_pages;
        const int64_t u0 = (r % pieces) * kUnits + threadIdx.x;
        const uint4* src = cache + (layer + from) * page_units;
        uint4* dst = cache + (layer + to) * page_units;
        uint4 x[kCopyUnits];
#pragma unroll
        for (int e = 0; e < kCopyUnits; ++e)
            if (u0 + e * kCopyThreads < page_units) x[e] = __ldcs(src + u0 + e * kCopyThreads);
#pragma unroll
        for (int e = 0; e < kCopyUnits; ++e)
            if (u0 + e * kCopyThreads < page_units) dst[u0 + e * kCopyThreads] = x[e];
    }
    if (retable && n > 0) {
        const int live = c.hdr->n_live;
        const int64_t entries = static_cast<int64_t>(c.n_seqs) * c.max_pages;
        for (int64_t x = static_cast<int64_t>(blockIdx.x) * kCopyThreads + threadIdx.x; x < entries;
             x += static_cast<int64_t>(gridDim.x) * kCopyThreads) {
            const int page = c.table[x];
            if (page >= live && page < c.n_pages) {
                const int to = c.pages[page];
                if (to >= 0) c.table[x] = to;
            }
        }
    }
}

// --------------------------------------------------------------------------------------- trim

__global__ void __launch_bounds__(256) trim_kernel(CacheArgs c, int64_t page_slots, int mult, int window,
                                                   int sinks) {
    const int64_t entries = static_cast<int64_t>(c.n_seqs) * c.max_pages;
    const int64_t x = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (x >= entries) return;
    const int64_t s = x / c.max_pages, e = x % c.max_pages;
    const int64_t keep_from = static_cast<int64_t>(c.lens[s]) * mult - window + 1;
    if (e * page_slots < sinks || (e + 1) * page_slots > keep_from) return;
    const int page = c.table[x];
    if (page < 0) return;
    c.table[x] = -1;
    if (page < c.n_pages) atomicSub(&c.refs[page], 1);
    else raise(c.status, DEV_BAD_PAGE);
}

cudaError_t sm_count(int& sms) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    return e != cudaSuccess ? e : cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
}

// The copy kernel, its launch overlapping the list kernel before it.
cudaError_t launch_copies(const CacheArgs& c, void* k_cache, void* v_cache, int n_layers,
                          size_t page_bytes, int retable, cudaStream_t stream) {
    int sms = 0;
    cudaError_t e = sm_count(sms);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(sms * (2048 / kCopyThreads));
    cfg.blockDim = dim3(kCopyThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, copy_pages_kernel, c, static_cast<uint4*>(k_cache),
                              static_cast<uint4*>(v_cache), n_layers,
                              static_cast<int64_t>(page_bytes / 16), retable);
}

}  // namespace

cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t stream) {
    int sms = 0;
    const cudaError_t e = sm_count(sms);
    if (e != cudaSuccess) return e;
    const int64_t units = static_cast<int64_t>(a.total) * a.row_units;
    const int64_t blocks = (units + kCopyThreads - 1) / kCopyThreads;
    const int64_t most = static_cast<int64_t>(sms) * (2048 / kCopyThreads) * 4;
    append_kernel<<<static_cast<unsigned>(blocks < most ? blocks : most), kCopyThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_cache_fork(const CacheArgs& c, const int32_t* src, const int32_t* dst, int n,
                              cudaStream_t stream) {
    share_kernel<true><<<1, kThreads, 0, stream>>>(c, src, dst, n);
    return cudaGetLastError();
}

cudaError_t launch_cache_free(const CacheArgs& c, const int32_t* seqs, int n, cudaStream_t stream) {
    share_kernel<false><<<1, kThreads, 0, stream>>>(c, nullptr, seqs, n);
    return cudaGetLastError();
}

cudaError_t launch_cache_reserve(const CacheArgs& c, const int32_t* seqs, const int32_t* new_tokens,
                                 int n, int page_shift, void* k_cache, void* v_cache, int n_layers,
                                 size_t page_bytes, cudaStream_t stream) {
    reserve_kernel<<<1, kThreads, 0, stream>>>(c, seqs, new_tokens, n, page_shift);
    const cudaError_t e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_copies(c, k_cache, v_cache, n_layers, page_bytes, 0, stream);
}

cudaError_t launch_cache_trim(const CacheArgs& c, int page_size, int window, int sinks, int mult,
                              cudaStream_t stream) {
    const int64_t entries = static_cast<int64_t>(c.n_seqs) * c.max_pages;
    trim_kernel<<<static_cast<unsigned>((entries + 255) / 256), 256, 0, stream>>>(
        c, static_cast<int64_t>(page_size) * mult, mult, window, sinks);
    return cudaGetLastError();
}

cudaError_t launch_cache_compact(const CacheArgs& c, void* k_cache, void* v_cache, int n_layers,
                                 size_t page_bytes, cudaStream_t stream) {
    compact_kernel<<<1, kThreads, 0, stream>>>(c);
    const cudaError_t e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_copies(c, k_cache, v_cache, n_layers, page_bytes, 1, stream);
}

}  // namespace pha
