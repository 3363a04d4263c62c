// pha_cache.cu -- the extern "C" boundary of the serving side (declared in include/pha_cache.h):
// argument checks, workspace layouts, launches.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/pha_cache.h"
#include "cache.cuh"
#include "gather.cuh"
#include "kernels.cuh"
#include "tensor_map.cuh"

using namespace pha;

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

size_t padded(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

// log2 of a power of two, -1 of anything else.
int log2_exact(int n) {
    if (n <= 0 || (n & (n - 1)) != 0) return -1;
    int s = 0;
    while ((1 << s) < n) ++s;
    return s;
}

pha_status of(cudaError_t e) { return e == cudaSuccess ? PHA_OK : PHA_ERR_CUDA; }

}  // namespace

extern "C" {

pha_status pha_cache_append(const void* k, const void* v, void* k_pages, void* v_pages,
                            const int32_t* page_table, int max_pages, int n_pages, int page_size,
                            const int32_t* cu_seqlens, const int32_t* kv_lens, int batch, int total,
                            int n_kv_heads, int head_dim, int element_bytes, int32_t* status,
                            pha_stream_t stream) {
    const int shift = log2_exact(page_size);
    if (batch <= 0 || total < 0 || max_pages <= 0 || n_pages <= 0 || n_kv_heads <= 0 || head_dim <= 0 ||
        shift < 0 || (element_bytes != 1 && element_bytes != 2 && element_bytes != 4) ||
        !aligned(status, 4))
        return PHA_ERR_INVALID;
    const int64_t row = static_cast<int64_t>(n_kv_heads) * head_dim * element_bytes;
    if (row % 16 != 0 || row > (1 << 30) ||
        (static_cast<int64_t>(n_pages) << shift) * n_kv_heads > INT32_MAX)
        return PHA_ERR_INVALID;
    if (total == 0) return PHA_OK;
    if (!k || !v || !k_pages || !v_pages || !page_table || !cu_seqlens || !kv_lens || !aligned(k, 16) ||
        !aligned(v, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(page_table, 4) ||
        !aligned(cu_seqlens, 4) || !aligned(kv_lens, 4))
        return PHA_ERR_INVALID;
    AppendArgs a{};
    a.k = static_cast<const uint4*>(k);
    a.v = static_cast<const uint4*>(v);
    a.k_pages = static_cast<uint4*>(k_pages);
    a.v_pages = static_cast<uint4*>(v_pages);
    a.table = page_table;
    a.cu = cu_seqlens;
    a.kv_lens = kv_lens;
    a.status = status;
    a.max_pages = max_pages;
    a.n_pages = n_pages;
    a.page_shift = shift;
    a.batch = batch;
    a.total = total;
    a.row_units = static_cast<int>(row / 16);
    return of(launch_cache_append(a, stream));
}

size_t pha_cache_workspace_bytes(int n_pages, int n_seqs) {
    if (n_pages <= 0 || n_seqs <= 0) return 0;
    const size_t seqs = padded(sizeof(int32_t) * static_cast<size_t>(n_seqs));
    const size_t pages = padded(sizeof(int32_t) * static_cast<size_t>(n_pages));
    return kWorkspaceHeaderBytes + 3 * seqs + 2 * (seqs > pages ? seqs : pages) + pages;
}

}  // extern "C"

namespace {

// Checks what the four workspace calls share and lays the workspace out. n: length of the lists.
pha_status cache_args(CacheArgs& c, int32_t* table, int max_pages, int32_t* lens, int n_seqs,
                      int32_t* refs, int n_pages, int n, void* workspace, size_t workspace_bytes,
                      int32_t* status) {
    if (!table || !refs || !aligned(table, 4) || !aligned(lens, 4) || !aligned(refs, 4) ||
        !aligned(status, 4) || max_pages <= 0 || n_seqs <= 0 || n_pages <= 0 || n < 0 || n > n_seqs)
        return PHA_ERR_INVALID;
    if (!workspace || !aligned(workspace, 16) ||
        workspace_bytes < pha_cache_workspace_bytes(n_pages, n_seqs))
        return PHA_ERR_WORKSPACE;
    c = CacheArgs{};
    c.table = table;
    c.lens = lens;
    c.refs = refs;
    c.status = status;
    c.max_pages = max_pages;
    c.n_seqs = n_seqs;
    c.n_pages = n_pages;
    const size_t seqs = padded(sizeof(int32_t) * static_cast<size_t>(n_seqs));
    const size_t pages = padded(sizeof(int32_t) * static_cast<size_t>(n_pages));
    const size_t both = seqs > pages ? seqs : pages;
    auto* w = static_cast<uint8_t*>(workspace);
    c.hdr = reinterpret_cast<CacheHeader*>(w);
    w += kWorkspaceHeaderBytes;
    c.marks = reinterpret_cast<int32_t*>(w);
    c.need = reinterpret_cast<int32_t*>(w + seqs);
    c.first = reinterpret_cast<int32_t*>(w + 2 * seqs);
    c.copy_src = reinterpret_cast<int32_t*>(w + 3 * seqs);
    c.copy_dst = reinterpret_cast<int32_t*>(w + 3 * seqs + both);
    c.pages = reinterpret_cast<int32_t*>(w + 3 * seqs + 2 * both);
    return PHA_OK;
}

bool bad_list(const int32_t* list, int n) { return n > 0 && (!list || !aligned(list, 4)); }

bool bad_pools(const void* k_cache, const void* v_cache, int n_layers, size_t page_bytes) {
    return !k_cache || !v_cache || !aligned(k_cache, 16) || !aligned(v_cache, 16) || n_layers <= 0 ||
           page_bytes == 0 || page_bytes % 16 != 0;
}

}  // namespace

extern "C" {

pha_status pha_cache_fork(int32_t* page_table, int max_pages, int32_t* kv_lens, int n_seqs,
                          int32_t* page_refs, int n_pages, const int32_t* src, const int32_t* dst,
                          int n, void* workspace, size_t workspace_bytes, int32_t* status,
                          pha_stream_t stream) {
    if (!kv_lens || bad_list(src, n) || bad_list(dst, n)) return PHA_ERR_INVALID;
    CacheArgs c;
    const pha_status st = cache_args(c, page_table, max_pages, kv_lens, n_seqs, page_refs, n_pages, n,
                                     workspace, workspace_bytes, status);
    return st != PHA_OK ? st : of(launch_cache_fork(c, src, dst, n, stream));
}

pha_status pha_cache_reserve(int32_t* page_table, int max_pages, int32_t* kv_lens, int n_seqs,
                             int32_t* page_refs, int n_pages, int page_size, const int32_t* seqs,
                             const int32_t* new_tokens, int n, void* k_cache, void* v_cache,
                             int n_layers, size_t page_bytes, void* workspace,
                             size_t workspace_bytes, int32_t* status, pha_stream_t stream) {
    const int shift = log2_exact(page_size);
    if (!kv_lens || bad_list(seqs, n) || bad_list(new_tokens, n) || shift < 0 ||
        bad_pools(k_cache, v_cache, n_layers, page_bytes))
        return PHA_ERR_INVALID;
    CacheArgs c;
    const pha_status st = cache_args(c, page_table, max_pages, kv_lens, n_seqs, page_refs, n_pages, n,
                                     workspace, workspace_bytes, status);
    return st != PHA_OK ? st : of(launch_cache_reserve(c, seqs, new_tokens, n, shift, k_cache, v_cache,
                                                       n_layers, page_bytes, stream));
}

pha_status pha_cache_free(int32_t* page_table, int max_pages, int32_t* kv_lens, int n_seqs,
                          int32_t* page_refs, int n_pages, const int32_t* seqs, int n,
                          void* workspace, size_t workspace_bytes, int32_t* status,
                          pha_stream_t stream) {
    if (!kv_lens || bad_list(seqs, n)) return PHA_ERR_INVALID;
    CacheArgs c;
    const pha_status st = cache_args(c, page_table, max_pages, kv_lens, n_seqs, page_refs, n_pages, n,
                                     workspace, workspace_bytes, status);
    return st != PHA_OK ? st : of(launch_cache_free(c, seqs, n, stream));
}

pha_status pha_cache_trim(int32_t* page_table, int max_pages, const int32_t* kv_lens, int n_seqs,
                          int32_t* page_refs, int n_pages, int page_size, int window, int sinks,
                          int paired, int32_t* status, pha_stream_t stream) {
    if (!page_table || !kv_lens || !page_refs || !aligned(page_table, 4) || !aligned(kv_lens, 4) ||
        !aligned(page_refs, 4) || !aligned(status, 4) || max_pages <= 0 || n_seqs <= 0 || n_pages <= 0 ||
        log2_exact(page_size) < 0 || window <= 0 || sinks < 0 || (paired != 0 && paired != 1) ||
        (static_cast<int64_t>(n_seqs) * max_pages + 255) / 256 > INT32_MAX)
        return PHA_ERR_INVALID;
    CacheArgs c{};
    c.table = page_table;
    c.lens = const_cast<int32_t*>(kv_lens);
    c.refs = page_refs;
    c.status = status;
    c.max_pages = max_pages;
    c.n_seqs = n_seqs;
    c.n_pages = n_pages;
    return of(launch_cache_trim(c, page_size, window, sinks, paired ? 2 : 1, stream));
}

pha_status pha_cache_compact(int32_t* page_table, int max_pages, int n_seqs, int32_t* page_refs,
                             int n_pages, void* k_cache, void* v_cache, int n_layers,
                             size_t page_bytes, void* workspace, size_t workspace_bytes,
                             int32_t* status, pha_stream_t stream) {
    if (bad_pools(k_cache, v_cache, n_layers, page_bytes)) return PHA_ERR_INVALID;
    CacheArgs c;
    const pha_status st = cache_args(c, page_table, max_pages, nullptr, n_seqs, page_refs, n_pages, 0,
                                     workspace, workspace_bytes, status);
    return st != PHA_OK ? st : of(launch_cache_compact(c, k_cache, v_cache, n_layers, page_bytes, stream));
}

}  // extern "C"

// ------------------------------------------------------------------------------ paged attention

namespace {

constexpr int kRowsSplitKeys = 1024;  // key columns of one warp's split (float32)
// Keys of a block of the decoding kernel, and what a block's start and its part of the join cost, in keys.
constexpr int kDecodeMinSplit = 512, kDecodeMaxSplit = 2048, kDecodeBlockCost = 300;

// Keys of a block, for `units` (sequence, kv head) pairs of up to `most` keys on `slots` blocks at a
// time: the ranges are equal and the number of them is the one whose rounds of blocks take least, counted
// as if every sequence had `most` keys. (Ranges of 2,048 keys whatever the rounds: 144 us instead of 68
// for 64 paired sequences of 3 slot heads and 4,106 keys.) At most kDecodeMaxSplit, so that long
// histories do not outlast the short ones' blocks.
int decode_split(int64_t units, int64_t slots, int64_t most) {
    int64_t best = 0, best_cost = INT64_MAX;
    const int64_t least = (most + kDecodeMaxSplit - 1) / kDecodeMaxSplit;
    for (int64_t n = least > 1 ? least : 1; n < least + 64; ++n) {
        const int64_t keys = ((most + n - 1) / n + 63) / 64 * 64;
        if (n > least && keys < kDecodeMinSplit) break;
        const int64_t cost = (units * n + slots - 1) / slots * (keys + kDecodeBlockCost);
        if (cost < best_cost) {
            best_cost = cost;
            best = keys;
        }
    }
    return static_cast<int>(best > kDecodeMinSplit ? best : kDecodeMinSplit);
}

struct PagedPlan {
    bool gather;                 // the tensor-core kernel with a plan
    bool decode;                 // few rows per sequence
    int window, sinks;           // as the kernels take them
    int n_splits, split_keys;
    int pack, tile_tokens, box_rows;
    int64_t tiles;
    GatherSpace space;
    size_t part_o, part_lse, bytes;  // workspace offsets
};

// The path, the splits and the workspace of a paged call. false: arguments out of range.
bool paged_plan(PagedPlan& w, int batch, int max_q, int max_kv, int total_q, int n_heads,
                int n_kv_heads, int head_dim, pha_dtype dtype, int window, int sinks, int paired,
                int page_size = 0) {
    if (batch <= 0 || max_q < 0 || max_kv < 0 || total_q < 0 || total_q > (1 << 28) ||
        max_kv > (1 << 29) || n_heads <= 0 || n_kv_heads <= 0 || n_heads > 4096 ||
        static_cast<int64_t>(total_q) * n_heads > INT32_MAX ||
        n_heads % n_kv_heads != 0 || head_dim <= 0 || head_dim > 128 || sinks < 0 ||
        (paired != 0 && paired != 1) || (paired && ((n_heads & 1) || (n_kv_heads & 1))))
        return false;
    w = PagedPlan{};
    const int mult = paired ? 2 : 1;
    const int heads = n_heads / mult, kv_heads = n_kv_heads / mult;
    // the most key columns the new tokens of one sequence can see
    int64_t most = static_cast<int64_t>(max_kv) * mult;
    w.window = window > 0 && window < most ? window : 0;  // a window past every cache hides nothing
    w.sinks = sinks < most ? sinks : static_cast<int>(most);
    window = w.window;
    sinks = w.sinks;
    if (window > 0) {
        const int64_t seen = static_cast<int64_t>(window) + static_cast<int64_t>(max_q) * mult + sinks;
        most = seen < most ? seen : most;
    }
    const int64_t rows_each = static_cast<int64_t>(max_q) * mult * (heads / kv_heads);
    w.decode = dtype == PHA_BF16 && rows_each <= kDecodeRows && batch <= 65535 && kv_heads <= 65535;
    w.gather = dtype == PHA_BF16 && !w.decode;
    if (w.gather) {
        // A TMA box stays in one page. Without a window columns begin at position 0 and it may be a whole
        // tile; with one they begin at a multiple of the box, so it is kept to 32 rows (16 of the
        // first tile's columns wasted on average).
        const int most_rows = window > 0 ? 32 : kBlockN;
        const int page_slots = page_size * mult;
        w.box_rows = page_slots < most_rows ? page_slots : most_rows;
        if (w.box_rows < 8) w.box_rows = 1;  // below the 8 rows of a swizzle pattern: gathered row by row
        w.pack = gather_pack(heads, kv_heads);
        w.tile_tokens = gather_tile_tokens(w.pack, window, sinks, most_rows);
        w.tiles = gather_tiles(batch, static_cast<int64_t>(max_q) * mult, static_cast<int64_t>(total_q) * mult,
                               w.tile_tokens);
        w.space = gather_space(batch, w.tiles, head_dim);
        w.part_o = w.space.part_o;
        w.part_lse = w.space.part_lse;
        w.bytes = w.space.bytes;
        return true;
    }
    // (no more splits than a grid's second dimension)
    w.split_keys = kRowsSplitKeys;
    while ((most + w.split_keys - 1) / w.split_keys > 65535) w.split_keys *= 2;
    if (w.decode) {
        // (blocks of 96 KB at hd 128, of 48 KB at hd 64)
        w.split_keys = decode_split(static_cast<int64_t>(batch) * kv_heads, kGatherCtas * (head_dim == 128 ? 2 : 4), most);
    }
    w.n_splits = static_cast<int>((most + w.split_keys - 1) / w.split_keys);
    if (w.n_splits < 1) w.n_splits = 1;
    const size_t rows = static_cast<size_t>(total_q) * n_heads;
    const size_t parts = w.n_splits > 1 ? rows * w.n_splits : 0;
    w.part_o = kWorkspaceHeaderBytes;
    w.part_lse = w.part_o + padded(parts * head_dim * sizeof(float));
    w.bytes = w.part_lse + padded(parts * sizeof(float));
    return true;
}

}  // namespace

extern "C" {

size_t pha_attn_paged_workspace_bytes(int batch, int max_q, int max_kv, int total_q, int n_heads,
                                      int n_kv_heads, int head_dim, pha_dtype dtype, int window,
                                      int sinks, int paired) {
    PagedPlan w;
    if (dtype != PHA_BF16 && dtype != PHA_F32) return 0;
    return paged_plan(w, batch, max_q, max_kv, total_q, n_heads, n_kv_heads, head_dim, dtype, window,
                      sinks, paired)
               ? w.bytes
               : 0;
}

}  // extern "C"

namespace {

// stall_us: test hook, see pha_test_attn_paged_fwd_stalled.
pha_status paged_fwd(const void* q, const void* k_pages, const void* v_pages,
                     const int32_t* page_table, int max_pages, int n_pages, int page_size,
                     const int32_t* cu_seqlens, const int32_t* kv_lens, int batch,
                     int max_q, int max_kv, int total_q, int n_heads, int n_kv_heads,
                     int head_dim, pha_dtype dtype, int window, int sinks, int paired,
                     float scale, void* o, float* lse, void* workspace,
                     size_t workspace_bytes, int32_t* status, pha_stream_t stream, int stall_us) {
    const int shift = log2_exact(page_size);
    if ((dtype != PHA_BF16 && dtype != PHA_F32) || shift < 0 || shift > 24 || n_pages <= 0 ||
        max_pages <= 0 || !(scale == scale) || !aligned(status, 4) || !aligned(lse, 4))
        return PHA_ERR_INVALID;
    if (head_dim > 128) return PHA_ERR_UNSUPPORTED;
    PagedPlan w;
    if (!paged_plan(w, batch, max_q, max_kv, total_q, n_heads, n_kv_heads, head_dim, dtype, window,
                    sinks, paired, page_size) ||
        (static_cast<int64_t>(n_pages) << shift) * n_kv_heads > INT32_MAX)
        return PHA_ERR_INVALID;
    if (dtype == PHA_BF16 && head_dim != 64 && head_dim != 128) return PHA_ERR_UNSUPPORTED;
    if (total_q == 0) return PHA_OK;
    if (!q || !k_pages || !v_pages || !o || !page_table || !cu_seqlens || !kv_lens || !aligned(q, 16) ||
        !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(o, 16) || !aligned(page_table, 4) ||
        !aligned(cu_seqlens, 4) || !aligned(kv_lens, 4))
        return PHA_ERR_INVALID;
    if (!workspace || !aligned(workspace, 16) || workspace_bytes < w.bytes) return PHA_ERR_WORKSPACE;
    if (stall_us != 0 && !w.gather) return PHA_ERR_UNSUPPORTED;  // (the other kernels have no waits)
    GatherProblem p{};
    p.test_stall_us = stall_us;
    p.q = q;
    p.k = k_pages;
    p.v = v_pages;
    p.o = o;
    p.lse = lse;
    p.cu = cu_seqlens;
    p.kv_lens = kv_lens;
    p.table = page_table;
    p.max_pages = max_pages;
    p.n_pages = n_pages;
    p.mult = paired ? 2 : 1;
    p.page_shift = shift + (paired ? 1 : 0);
    p.batch = batch;
    p.max_q = max_q;
    p.max_kv = max_kv;
    p.total_q = total_q;
    p.heads = n_heads / p.mult;
    p.kv_heads = n_kv_heads / p.mult;
    p.head_dim = head_dim;
    p.window = w.window;
    p.sinks = w.sinks;
    p.scale = scale > 0.f ? scale : 1.0f / sqrtf(static_cast<float>(head_dim));
    p.n_splits = w.n_splits;
    p.split_keys = w.split_keys;
    auto* base = static_cast<uint8_t*>(workspace);
    p.part_o = reinterpret_cast<float*>(base + w.part_o);
    p.part_lse = reinterpret_cast<float*>(base + w.part_lse);
    p.status = status;
    if (!w.gather) {
        cudaError_t e = w.decode ? launch_attn_decode(p, stream) : launch_attn_rows(p, stream);
        if (e == cudaSuccess && p.n_splits > 1) e = launch_attn_join(p, w.decode, stream);
        return of(e);
    }
    p.hdr = reinterpret_cast<WorkspaceHeader*>(base);
    p.tiles = reinterpret_cast<int4*>(base + w.space.tiles);
    p.starts = reinterpret_cast<int4*>(base + w.space.starts);
    p.n_cta = kGatherCtas;
    p.pack = w.pack;
    p.tile_tokens = w.tile_tokens;
    p.box_rows = w.box_rows;
    CUtensorMap tq, tk, tv;
    const uint64_t rows = static_cast<uint64_t>(n_pages) << p.page_shift;
    const uint64_t width = static_cast<uint64_t>(p.kv_heads) * head_dim;
    const uint32_t box = w.box_rows < 8 ? 8 : w.box_rows;  // (below 8 the maps are not used)
    if (!encode_pack_map(&tq, q, head_dim, p.heads, static_cast<uint64_t>(total_q) * p.mult,
                         128 % p.pack == 0 ? p.pack : 1) ||
        !encode_slot_map(&tk, k_pages, width, rows, box) || !encode_slot_map(&tv, v_pages, width, rows, box))
        return PHA_ERR_CUDA;
    if (launch_gather_plan(p, w.tiles, reinterpret_cast<int*>(base + w.space.before),
                           reinterpret_cast<int64_t*>(base + w.space.steps), false, stream) != cudaSuccess)
        return PHA_ERR_CUDA;
    if (w.tiles == 0) return PHA_OK;  // no new tokens are allowed for: the plan has checked the lengths
    return of(launch_attn_gather(p, tq, tk, tv, tk, tv, stream));
}

}  // namespace

extern "C" {

pha_status pha_attn_paged_fwd(const void* q, const void* k_pages, const void* v_pages,
                              const int32_t* page_table, int max_pages, int n_pages, int page_size,
                              const int32_t* cu_seqlens, const int32_t* kv_lens, int batch,
                              int max_q, int max_kv, int total_q, int n_heads, int n_kv_heads,
                              int head_dim, pha_dtype dtype, int window, int sinks, int paired,
                              float scale, void* o, float* lse, void* workspace,
                              size_t workspace_bytes, int32_t* status, pha_stream_t stream) {
    return paged_fwd(q, k_pages, v_pages, page_table, max_pages, n_pages, page_size, cu_seqlens, kv_lens, batch,
                     max_q, max_kv, total_q, n_heads, n_kv_heads, head_dim, dtype, window, sinks, paired, scale, o,
                     lse, workspace, workspace_bytes, status, stream, 0);
}

pha_status pha_test_attn_paged_fwd_stalled(const void* q, const void* k_pages, const void* v_pages,
                                           const int32_t* page_table, int max_pages, int n_pages,
                                           int page_size, const int32_t* cu_seqlens,
                                           const int32_t* kv_lens, int batch, int max_q, int max_kv,
                                           int total_q, int n_heads, int n_kv_heads, int head_dim,
                                           pha_dtype dtype, int window, int sinks, int paired,
                                           float scale, void* o, float* lse, void* workspace,
                                           size_t workspace_bytes, int32_t* status, int stall_us,
                                           pha_stream_t stream) {
    if (stall_us < 1 || stall_us > 100000) return PHA_ERR_INVALID;
    return paged_fwd(q, k_pages, v_pages, page_table, max_pages, n_pages, page_size, cu_seqlens, kv_lens, batch,
                     max_q, max_kv, total_q, n_heads, n_kv_heads, head_dim, dtype, window, sinks, paired, scale, o,
                     lse, workspace, workspace_bytes, status, stream, stall_us);
}

}  // extern "C"
