// gather.cuh -- what the attention kernels of the streaming mask share: the problem, a sequence's
// place in it, and which keys a row of queries sees.
//
// A query at position p of its sequence sees key position j iff j <= p and (p - j < window or
// j < sinks) (window 0: every j <= p). For a run of queries at positions [p0, p0 + n) the keys that
// some of them see are listed as columns c = 0, 1, ...: first the window part, positions
// [lo, p0 + n) with lo = max(0, p0 - window + 1), then the sinks below it, positions [0, min(sinks,
// lo)). The kernels gather the rows of these columns by themselves (through the page table, or from
// the packed documents), so keys that nobody sees are neither read nor multiplied, and the sinks
// share the last tile with the end of the window instead of taking a tile of their own.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kernels.cuh"

namespace pha {

struct GatherProblem {
    const void* q;
    const void* k;
    const void* v;
    void* o;
    float* lse;
    const int32_t* cu;       // [batch + 1] rows of q, tokens
    const int32_t* kv_lens;  // paged: tokens in the cache; NULL: keys are the packed documents
    const int32_t* table;    // paged: [batch][max_pages]
    int max_pages, n_pages;
    int page_shift;          // log2 of the slots of a page
    int batch, max_q, max_kv, total_q;  // tokens
    int mult;                // slots per token (2 paired)
    int heads, kv_heads, head_dim;      // of the slot view
    int window, sinks;
    float scale;
    // Partial results: normalised o (float32) and log2 of the sum of exponentials. CUDA cores and single
    // tokens: [split][q slot][head], split s having columns [s, s + 1) * split_keys of its sequence
    // (a sequence with one split writes o itself). Tensor cores: [2 per CTA][row of the tile].
    int n_splits, split_keys;
    float* part_o;
    float* part_lse;
    int32_t* status;         // may be NULL
    // Plan of the tensor-core kernel (gather_plan.cu): its header, which also holds the device status
    // of a call with one (NULL: none), the row tiles and where each CTA's share begins.
    WorkspaceHeader* hdr;
    int4* tiles;
    int4* starts;
    int n_cta;               // CTAs that share the work
    // Tensor cores: a row of a query tile is (token, head) with `pack` heads of one kv head's group
    // side by side (rows r = token * pack + head), tile_tokens tokens a row tile.
    int pack, tile_tokens;
    int box_rows;            // rows of a TMA box over k / v; paged: they lie in one page, and columns
                             // begin at multiples of it (1: no TMA)
    int test_stall_us;       // test hook: > 0 makes the softmax warps wait that long for nothing
};

// One row tile: up to 256 rows (two sub-tiles) of one sequence, times each chunk of `pack` heads.
//   x = first q slot, y = tokens | keys of the sequence behind the tile's last (at most 127) << 16,
//   z = position of the first token, w = sequence (paged) or slot of key 0 (documents).
// The work of all (row tile, chunk) items lies on one line, key tile by key tile with one step more
// per item for its fixed costs, and is cut into n_cta equal shares: starts[c] = (row tile, chunk, key
// tile) where CTA c begins. Items that a cut divides leave partial rows, which attn_join_cuts joins.
constexpr int kGatherRows = 2 * kBlockM;

struct GatherSeq {
    int64_t q0;    // first q slot
    int n_q, kv;   // query and key slots
    int64_t base;  // documents: slot of key 0
    bool ok;
};

__device__ __forceinline__ GatherSeq gather_seq(const GatherProblem& p, int b) {
    GatherSeq s;
    const int64_t a = __ldg(p.cu + b), z = __ldg(p.cu + b + 1);
    const int64_t n = z - a;
    int64_t kv = n;
    s.ok = a >= 0 && n >= 0 && z <= p.total_q && n <= p.max_q;
    if (p.kv_lens) {
        kv = __ldg(p.kv_lens + b);
        s.ok = s.ok && (n == 0 || (kv >= n && kv <= p.max_kv &&
                                   kv * p.mult <= static_cast<int64_t>(p.max_pages) << p.page_shift));
    }
    s.q0 = a * p.mult;
    s.n_q = s.ok ? static_cast<int>(n) * p.mult : 0;
    s.kv = s.ok ? static_cast<int>(kv) * p.mult : 0;
    s.base = p.kv_lens ? 0 : s.q0;
    return s;
}

// The columns of the queries at positions [p0, p0 + n).
struct GatherCols {
    int lo;      // position of column 0
    int n_w;     // columns of the window part
    int total;   // all columns
};

// align (a power of two): lo is rounded down to a multiple of it.
__device__ __forceinline__ GatherCols gather_cols(const GatherProblem& p, int p0, int n, int align = 1) {
    GatherCols c;
    c.lo = (p.window > 0 && p0 - p.window + 1 > 0) ? (p0 - p.window + 1) & ~(align - 1) : 0;
    c.n_w = p0 + n - c.lo;
    c.total = c.n_w + (p.sinks < c.lo ? p.sinks : c.lo);
    return c;
}

// Position of column col.
__device__ __forceinline__ int col_pos(const GatherCols& c, int col) {
    return col < c.n_w ? c.lo + col : col - c.n_w;
}

// Whether a query at position pos sees column col (< total).
__device__ __forceinline__ bool col_visible(const GatherProblem& p, const GatherCols& c, int col, int pos) {
    if (col >= c.n_w) return true;  // a sink below everyone's window
    const int j = c.lo + col;
    return j <= pos && (p.window <= 0 || pos - j < p.window || j < p.sinks);
}

// Row of k / v (in rows of kv_heads * head_dim) of key position pos of sequence b; -1 when the page
// table has no page there.
template <bool PAGED>
__device__ __forceinline__ int64_t key_row(const GatherProblem& p, int b, int64_t base, int pos) {
    if (!PAGED) return base + pos;
    const int page = __ldg(p.table + static_cast<int64_t>(b) * p.max_pages + (pos >> p.page_shift));
    if (page < 0 || page >= p.n_pages) return -1;
    return (static_cast<int64_t>(page) << p.page_shift) + (pos & ((1 << p.page_shift) - 1));
}

// Last sequence whose first row is at or before token t (-1: none).
__device__ __forceinline__ int gather_seq_of(const int32_t* __restrict__ cu, int batch, int t) {
    int lo = -1, hi = batch;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(cu + mid) <= t) lo = mid; else hi = mid;
    }
    return lo;
}

// Heads of a group that share a query tile: all of them, or one at a time when they would not fit a
// sub-tile.
inline int gather_pack(int heads, int kv_heads) {
    const int g = heads / kv_heads;
    return g <= kBlockM ? g : 1;
}

// Columns of a tile's first key are aligned to this (see box_rows).
__host__ __device__ inline int gather_align(bool paged, int box_rows) { return paged ? box_rows : 1; }

// Tokens of a row tile: as many as fit its rows, or fewer where that saves a whole key tile and the
// rows per key tile go up. (A run of T tokens sees window + T - 1 + sinks columns, so with a window
// of a multiple of 128 the last tile would hold a few columns only.)
inline int gather_tile_tokens(int pack, int window, int sinks, int align) {
    const int most = kGatherRows / pack;
    if (window <= 0) return most;
    const int64_t fixed = static_cast<int64_t>(window) - 1 + (align - 1) + sinks;
    const int64_t tiles = (fixed + most + kBlockN - 1) / kBlockN;
    const int64_t fewer = (tiles - 1) * kBlockN - fixed;
    return fewer >= 1 && fewer * tiles > most * (tiles - 1) ? static_cast<int>(fewer) : most;
}

// Bound on the row tiles of a call.
inline int64_t gather_tiles(int batch, int64_t max_q, int64_t total_q, int tile_tokens) {
    const int64_t per_seq = (max_q + tile_tokens - 1) / tile_tokens;
    const int64_t by_rows = total_q / tile_tokens + batch;
    return per_seq > by_rows / batch ? by_rows : per_seq * batch;  // (their product may pass 63 bits)
}

constexpr int kGatherCtas = 148;      // SMs of a B200; workspaces may not depend on the device at hand
constexpr int kGatherMinSteps = 3;    // key tiles (and item costs) of a CTA's share, at least

// Workspace of the plan and the partial rows, from byte 0 (the header).
struct GatherSpace {
    size_t before, steps, tiles, starts, part_o, part_lse, bytes;
};
inline GatherSpace gather_space(int batch, int64_t tiles, int head_dim) {
    const auto padded = [](size_t n) { return (n + 255) & ~static_cast<size_t>(255); };
    GatherSpace w;
    w.before = kWorkspaceHeaderBytes;
    w.steps = w.before + padded(sizeof(int) * (static_cast<size_t>(batch) + 1));
    w.tiles = w.steps + padded(sizeof(int64_t) * (static_cast<size_t>(tiles) + 1));
    w.starts = w.tiles + padded(sizeof(int4) * static_cast<size_t>(tiles));
    w.part_o = w.starts + padded(sizeof(int4) * (kGatherCtas + 1));
    const size_t rows = 2 * static_cast<size_t>(kGatherCtas) * kGatherRows;
    w.part_lse = w.part_o + rows * head_dim * sizeof(float);
    w.bytes = w.part_lse + rows * sizeof(float);
    return w;
}

// Checks the lengths and lays out the work (max_tiles 0: the check alone). strict: any bad length
// makes the plan empty (header status 1); otherwise only the bad sequences are left out (p.status 1).
// before: int[batch + 1], steps: int64[max_tiles + 1].
cudaError_t launch_gather_plan(const GatherProblem& p, int64_t max_tiles, int* before, int64_t* steps,
                               bool strict, cudaStream_t stream);

// bf16, head_dim 64 / 128, on the tensor cores, by the plan; then the cut items. tm_q: encode_pack_map
// over q (used when pack divides 128); tm_k, tm_v: maps over the rows of k / v, 64 x box_rows boxes; tm_k8,
// tm_v8: the same with boxes of 8 rows (documents; not used for pages).
cudaError_t launch_attn_gather(const GatherProblem& p, const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                               const CUtensorMap& tm_v, const CUtensorMap& tm_k8, const CUtensorMap& tm_v8,
                               cudaStream_t stream);

// bf16, head_dim 64 / 128, few rows: at most kDecodeRows (new slots times a group's heads) a sequence, the
// rows of its products; block per (split, kv head, sequence). (This and the row tiles of attn_gather.cu, us:
// 64 ragged histories, 32 / 8 heads of 128, 4, 8 and 16 rows: 185 / 234, 178 / 220, 213 / 254; 32 paired
// streams of window 4,096, 2, 8 and 16 rows: 43 / 67, 46 / 68, 47 / 72.)
constexpr int kDecodeRows = 16;
cudaError_t launch_attn_decode(const GatherProblem& p, cudaStream_t stream);

// float32 on CUDA cores: one warp per (row, split).
cudaError_t launch_attn_rows(const GatherProblem& p, cudaStream_t stream);

// Joins the splits of every row into o and lse.
cudaError_t launch_attn_join(const GatherProblem& p, int is_bf16, cudaStream_t stream);

}  // namespace pha
