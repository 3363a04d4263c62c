// pha_sinks.cu -- the extern "C" boundary of attention with a sliding window and sinks (declared in
// include/pha_sinks.h): argument checks, workspace layouts, launches.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/pha_sinks.h"
#include "gather.cuh"
#include "kernels.cuh"
#include "tensor_map.cuh"

using namespace pha;

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

pha_status of(cudaError_t e) { return e == cudaSuccess ? PHA_OK : PHA_ERR_CUDA; }

constexpr int kMostTokens = 1 << 29;

// Shape checks of both directions. (batch times the longest document is bounded so that workspace sizes, which
// grow with it, fit 64 bits.)
pha_status shape_status(int batch, int max_len, int total_tokens, int n_heads, int n_kv_heads,
                        int head_dim, pha_dtype dtype, int sinks, int paired, float scale) {
    if ((dtype != PHA_BF16 && dtype != PHA_F32) || batch <= 0 || max_len < 0 || total_tokens < 0 ||
        total_tokens > kMostTokens || n_heads <= 0 || n_kv_heads <= 0 || n_heads > 4096 ||
        static_cast<int64_t>(total_tokens) * n_heads > INT32_MAX ||
        static_cast<int64_t>(batch) * (max_len < kMostTokens ? max_len : kMostTokens) > static_cast<int64_t>(1) << 48 ||
        n_heads % n_kv_heads != 0 || head_dim <= 0 || sinks < 0 || (paired != 0 && paired != 1) ||
        !(scale == scale) || (paired && ((n_heads & 1) || (n_kv_heads & 1))))
        return PHA_ERR_INVALID;
    if (sinks > kBlockN || head_dim > 128 || (dtype == PHA_BF16 && head_dim != 64 && head_dim != 128))
        return PHA_ERR_UNSUPPORTED;
    return PHA_OK;
}

// No document is longer than the rows there are, however loose the bound max_len.
int longest(int max_len, int total_tokens) { return max_len < total_tokens ? max_len : total_tokens; }

// A window that reaches past the longest document hides nothing: no window (0), as the kernels' index
// arithmetic wants it.
int real_window(int window, int max_len, int paired) {
    return window > 0 && window < static_cast<int64_t>(max_len) * (paired ? 2 : 1) ? window : 0;
}

size_t padded(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

// Forward: row tiles, and tokens of one (documents of any lengths up to max_len).
struct FwdPlan {
    int pack, tile_tokens;
    int64_t tiles;
    GatherSpace space;
};

FwdPlan fwd_plan(int batch, int max_len, int n_heads, int n_kv_heads, int head_dim, int window, int sinks,
                 int paired) {
    const int mult = paired ? 2 : 1;
    max_len = longest(max_len, kMostTokens);
    const int64_t slots = static_cast<int64_t>(max_len) * mult;
    FwdPlan w;
    w.pack = gather_pack(n_heads / mult, n_kv_heads / mult);
    w.tile_tokens = gather_tile_tokens(w.pack, real_window(window, max_len, paired), sinks, 1);
    w.tiles = gather_tiles(batch, slots, slots * batch, w.tile_tokens);
    w.space = gather_space(batch, w.tiles, head_dim);
    return w;
}

// Backward: header, per-document scratch and work list of the query tiles, the same of the key tiles
// (with far pieces; apart, so that a later call over the same documents keeps both lists), D (or -D),
// -lse log2(e), the far pieces' partial sums. Every document's last tile and last piece may be ragged: at most
// one of each more than whole ones fit.
struct BwdPlan {
    int64_t items_q, items_k;
    size_t list, keys, dsum, nlse, part, bytes;  // list: of a work list behind its header
};

BwdPlan bwd_plan(int batch, int max_len, int total_tokens, int n_heads, int n_kv_heads, int head_dim,
                 int window, int sinks, int paired) {
    const int mult = paired ? 2 : 1;
    const int64_t slots = static_cast<int64_t>(total_tokens) * mult;
    max_len = longest(max_len, total_tokens);
    window = real_window(window, max_len, paired);
    const bool far = window > 0 && sinks > 0;
    const int piece = far ? sink_piece_tiles(window, max_len, mult) : 1;
    // (documents of up to max_len, as long as the rows last)
    const auto items = [&](int64_t rows) {
        const int64_t each = (static_cast<int64_t>(max_len) * mult + rows - 1) / rows, all = slots / rows + batch;
        return each > all / batch ? all : each * batch;
    };
    const int64_t tiles = items(kBlockN), pieces = far ? items(static_cast<int64_t>(piece) * kBlockN) : 0;
    BwdPlan w{};
    w.items_q = tiles * (n_heads / mult);
    w.items_k = (tiles + pieces) * (n_heads / mult);
    w.list = kWorkspaceHeaderBytes + workspace_doc_bytes(batch);
    w.keys = padded(w.list + sizeof(int4) * static_cast<size_t>(w.items_q));
    w.dsum = w.keys + padded(w.list + sizeof(int4) * static_cast<size_t>(w.items_k));
    w.nlse = w.dsum + padded(sizeof(float) * static_cast<size_t>(total_tokens) * n_heads);
    w.part = w.nlse + padded(sizeof(float) * static_cast<size_t>(total_tokens) * n_heads);
    w.bytes = w.part + (far ? padded(sizeof(float) * static_cast<size_t>(sink_part_slots(batch, slots, piece)) *
                                     (n_kv_heads / mult) * sinks * 2 * head_dim)
                            : 0);
    return w;
}

}  // namespace

extern "C" {

size_t pha_attn_sinks_workspace_bytes(int batch, int max_len, int n_heads, int n_kv_heads,
                                      int head_dim, int window, int sinks, int paired) {
    if (shape_status(batch, max_len, 0, n_heads, n_kv_heads, head_dim, PHA_F32, sinks, paired, 0.f) != PHA_OK)
        return 0;
    return fwd_plan(batch, max_len, n_heads, n_kv_heads, head_dim, window, sinks, paired).space.bytes;
}

size_t pha_attn_sinks_bwd_workspace_bytes(int batch, int max_len, int total_tokens, int n_heads,
                                          int n_kv_heads, int head_dim, int window, int sinks,
                                          int paired) {
    if (shape_status(batch, max_len, total_tokens, n_heads, n_kv_heads, head_dim, PHA_F32, sinks, paired,
                     0.f) != PHA_OK)
        return 0;
    return bwd_plan(batch, max_len, total_tokens, n_heads, n_kv_heads, head_dim, window, sinks, paired).bytes;
}

}  // extern "C"

namespace {

// stall_us: test hook, see pha_test_attn_sinks_fwd_stalled.
pha_status sinks_fwd(const void* q, const void* k, const void* v,
                     const int32_t* cu_seqlens, int batch, int max_len, int total_tokens,
                     int n_heads, int n_kv_heads, int head_dim, pha_dtype dtype,
                     int window, int sinks, int paired, float scale, void* o, float* lse,
                     void* workspace, size_t workspace_bytes, pha_stream_t stream, int stall_us) {
    const pha_status st = shape_status(batch, max_len, total_tokens, n_heads, n_kv_heads, head_dim, dtype,
                                       sinks, paired, scale);
    if (st != PHA_OK) return st;
    const bool have = total_tokens > 0;
    if ((have && (!q || !k || !v || !o || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) ||
                  !aligned(o, 16))) ||
        !cu_seqlens || !aligned(cu_seqlens, 4) || !aligned(lse, 4))
        return PHA_ERR_INVALID;
    if (!workspace || !aligned(workspace, 16) ||
        workspace_bytes < pha_attn_sinks_workspace_bytes(batch, max_len, n_heads, n_kv_heads, head_dim,
                                                         window, sinks, paired))
        return PHA_ERR_WORKSPACE;
    GatherProblem p{};
    p.test_stall_us = stall_us;
    p.q = q;
    p.k = k;
    p.v = v;
    p.o = o;
    p.lse = lse;
    p.cu = cu_seqlens;
    p.batch = batch;
    p.max_q = p.max_kv = max_len;
    p.total_q = total_tokens;
    p.mult = paired ? 2 : 1;
    p.heads = n_heads / p.mult;
    p.kv_heads = n_kv_heads / p.mult;
    p.head_dim = head_dim;
    p.window = real_window(window, longest(max_len, total_tokens), paired);
    p.sinks = sinks;
    p.scale = scale > 0.f ? scale : 1.0f / sqrtf(static_cast<float>(head_dim));
    const FwdPlan w = fwd_plan(batch, max_len, n_heads, n_kv_heads, head_dim, window, sinks, paired);
    auto* base = static_cast<uint8_t*>(workspace);
    p.hdr = reinterpret_cast<WorkspaceHeader*>(base);
    p.tiles = reinterpret_cast<int4*>(base + w.space.tiles);
    p.starts = reinterpret_cast<int4*>(base + w.space.starts);
    p.part_o = reinterpret_cast<float*>(base + w.space.part_o);
    p.part_lse = reinterpret_cast<float*>(base + w.space.part_lse);
    p.n_cta = kGatherCtas;
    p.pack = w.pack;
    p.tile_tokens = w.tile_tokens;
    p.box_rows = kBlockN;
    const bool tc = dtype == PHA_BF16;
    if (launch_gather_plan(p, tc ? w.tiles : 0, reinterpret_cast<int*>(base + w.space.before),
                           reinterpret_cast<int64_t*>(base + w.space.steps), true, stream) != cudaSuccess)
        return PHA_ERR_CUDA;
    if (!have || max_len == 0) return PHA_OK;
    if (!tc) return of(launch_attn_rows(p, stream));
    CUtensorMap tq, tk, tv, tk8, tv8;
    const uint64_t rows = static_cast<uint64_t>(total_tokens) * p.mult;
    const uint64_t width = static_cast<uint64_t>(p.kv_heads) * head_dim;
    if (!encode_pack_map(&tq, q, head_dim, p.heads, rows, 128 % p.pack == 0 ? p.pack : 1) ||
        !encode_slot_map(&tk, k, width, rows) || !encode_slot_map(&tv, v, width, rows) ||
        !encode_slot_map(&tk8, k, width, rows, 8) || !encode_slot_map(&tv8, v, width, rows, 8))
        return PHA_ERR_CUDA;
    return of(launch_attn_gather(p, tq, tk, tv, tk8, tv8, stream));
}

pha_status sinks_bwd(const void* q, const void* k, const void* v, const void* o,
                     const float* lse, const void* dout, const int32_t* cu_seqlens,
                     int batch, int max_len, int total_tokens, int n_heads,
                     int n_kv_heads, int head_dim, pha_dtype dtype, int window, int sinks,
                     int paired, float scale, void* dq, void* dk, void* dv,
                     void* workspace, size_t workspace_bytes, pha_stream_t stream, int stall_us) {
    const pha_status st = shape_status(batch, max_len, total_tokens, n_heads, n_kv_heads, head_dim, dtype,
                                       sinks, paired, scale);
    if (st != PHA_OK) return st;
    const bool have = total_tokens > 0;
    if ((have && (!q || !k || !v || !o || !lse || !dout || !dq || !dk || !dv || !aligned(q, 16) ||
                  !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(dout, 16) ||
                  !aligned(dq, 16) || !aligned(dk, 16) || !aligned(dv, 16) || !aligned(lse, 4))) ||
        !cu_seqlens || !aligned(cu_seqlens, 4))
        return PHA_ERR_INVALID;
    if (!have) return PHA_OK;  // nothing to do (no launch, the workspace is not touched)
    if (!workspace || !aligned(workspace, 16) ||
        workspace_bytes < pha_attn_sinks_bwd_workspace_bytes(batch, max_len, total_tokens, n_heads,
                                                             n_kv_heads, head_dim, window, sinks, paired))
        return PHA_ERR_WORKSPACE;
    AttnProblem p{};
    p.test_stall_us = stall_us;
    p.q = q;
    p.k = k;
    p.v = v;
    p.cu_seqlens = cu_seqlens;
    p.batch = batch;
    p.max_len = longest(max_len, total_tokens);
    p.total_tokens = total_tokens;
    p.slot_mult = paired ? 2 : 1;
    p.heads = n_heads / p.slot_mult;
    p.kv_heads = n_kv_heads / p.slot_mult;
    p.head_dim = head_dim;
    p.causal = 1;
    p.window = real_window(window, p.max_len, paired);
    p.sinks = p.window > 0 ? sinks : 0;
    p.scale = scale > 0.f ? scale : 1.0f / sqrtf(static_cast<float>(head_dim));
    p.lse = const_cast<float*>(lse);
    const BwdPlan w = bwd_plan(batch, max_len, total_tokens, n_heads, n_kv_heads, head_dim, window, sinks, paired);
    auto* base = static_cast<uint8_t*>(workspace);
    auto* hdr = reinterpret_cast<WorkspaceHeader*>(base);
    auto* hdr_k = reinterpret_cast<WorkspaceHeader*>(base + w.keys);
    auto list = [&](size_t at) { return reinterpret_cast<int4*>(base + at + w.list); };
    auto build = [&](ScheduleMode mode, size_t at, int64_t items, bool beside) {
        return launch_schedule(p, mode, items < INT32_MAX ? static_cast<int>(items) : INT32_MAX,
                               reinterpret_cast<int*>(base + at + kWorkspaceHeaderBytes), list(at),
                               reinterpret_cast<WorkspaceHeader*>(base + at), stream, beside);
    };
    float* dsum = reinterpret_cast<float*>(base + w.dsum);
    p.sink_part = reinterpret_cast<float*>(base + w.part);
    p.checked = hdr;
    const bool tc = dtype == PHA_BF16;
    if (!tc) {
        // the scheduler also checks cu_seqlens; without a list to walk (CUDA cores) only that is used
        if (build(kSchedTilesQ, 0, w.items_q, false) != cudaSuccess) return PHA_ERR_CUDA;
        if (launch_attn_bwd_dsum(p, o, dout, dsum, 0, stream) != cudaSuccess) return PHA_ERR_CUDA;
        return of(launch_attn_bwd(p, dout, dsum, dq, dk, dv, 0, stream));
    }
    float* nlse = reinterpret_cast<float*>(base + w.nlse);
    const uint64_t rows = static_cast<uint64_t>(total_tokens) * p.slot_mult;
    const uint64_t wq = static_cast<uint64_t>(p.heads) * head_dim, wk = static_cast<uint64_t>(p.kv_heads) * head_dim;
    CUtensorMap tq, tk, tv, tdo, tdq, tdk, tdv;
    if (!encode_slot_map(&tq, q, wq, rows) || !encode_slot_map(&tk, k, wk, rows) ||
        !encode_slot_map(&tv, v, wk, rows) || !encode_slot_map(&tdo, dout, wq, rows) ||
        !encode_slot_map(&tdq, dq, wq, rows, 32) || !encode_slot_map(&tdk, dk, wk, rows, 16) ||
        !encode_slot_map(&tdv, dv, wk, rows, 16))
        return PHA_ERR_CUDA;
    // both lists and the rows' sums at the same time
    if (launch_attn_bwd_zero_outside(p, dq, dk, dv, stream) != cudaSuccess ||
        build(kSchedTilesQ, 0, w.items_q, false) != cudaSuccess ||
        build(kSchedTilesK, w.keys, w.items_k, true) != cudaSuccess ||
        launch_attn_bwd_sinks_rows(p, o, dout, nlse, dsum, stream) != cudaSuccess ||
        launch_attn_bwd_sinks_dq(p, tq, tk, tv, tdo, tdq, nlse, dsum, dq, list(0), hdr, &hdr->status,
                                 stream) != cudaSuccess)
        return PHA_ERR_CUDA;
    return of(launch_attn_bwd_sinks_dkdv(p, tq, tk, tv, tdo, tdk, tdv, nlse, dsum, dk, dv, list(w.keys), hdr_k,
                                         &hdr->status, stream));  // (one status word for the call)
}

pha_status stall_status(int stall_us, pha_dtype dtype) {
    if (stall_us < 1 || stall_us > 100000) return PHA_ERR_INVALID;
    return dtype == PHA_F32 ? PHA_ERR_UNSUPPORTED : PHA_OK;
}

}  // namespace

extern "C" {

pha_status pha_attn_sinks_fwd(const void* q, const void* k, const void* v,
                              const int32_t* cu_seqlens, int batch, int max_len, int total_tokens,
                              int n_heads, int n_kv_heads, int head_dim, pha_dtype dtype,
                              int window, int sinks, int paired, float scale, void* o, float* lse,
                              void* workspace, size_t workspace_bytes, pha_stream_t stream) {
    return sinks_fwd(q, k, v, cu_seqlens, batch, max_len, total_tokens, n_heads, n_kv_heads, head_dim, dtype,
                     window, sinks, paired, scale, o, lse, workspace, workspace_bytes, stream, 0);
}

pha_status pha_attn_sinks_bwd(const void* q, const void* k, const void* v, const void* o,
                              const float* lse, const void* dout, const int32_t* cu_seqlens,
                              int batch, int max_len, int total_tokens, int n_heads,
                              int n_kv_heads, int head_dim, pha_dtype dtype, int window, int sinks,
                              int paired, float scale, void* dq, void* dk, void* dv,
                              void* workspace, size_t workspace_bytes, pha_stream_t stream) {
    return sinks_bwd(q, k, v, o, lse, dout, cu_seqlens, batch, max_len, total_tokens, n_heads, n_kv_heads,
                     head_dim, dtype, window, sinks, paired, scale, dq, dk, dv, workspace, workspace_bytes,
                     stream, 0);
}

pha_status pha_test_attn_sinks_fwd_stalled(const void* q, const void* k, const void* v,
                                           const int32_t* cu_seqlens, int batch, int max_len,
                                           int total_tokens, int n_heads, int n_kv_heads,
                                           int head_dim, pha_dtype dtype, int window, int sinks,
                                           int paired, float scale, void* o, float* lse,
                                           void* workspace, size_t workspace_bytes, int stall_us,
                                           pha_stream_t stream) {
    const pha_status st = stall_status(stall_us, dtype);
    return st != PHA_OK ? st
                        : sinks_fwd(q, k, v, cu_seqlens, batch, max_len, total_tokens, n_heads, n_kv_heads,
                                    head_dim, dtype, window, sinks, paired, scale, o, lse, workspace,
                                    workspace_bytes, stream, stall_us);
}

pha_status pha_test_attn_sinks_bwd_stalled(const void* q, const void* k, const void* v,
                                           const void* o, const float* lse, const void* dout,
                                           const int32_t* cu_seqlens, int batch, int max_len,
                                           int total_tokens, int n_heads, int n_kv_heads,
                                           int head_dim, pha_dtype dtype, int window, int sinks,
                                           int paired, float scale, void* dq, void* dk, void* dv,
                                           void* workspace, size_t workspace_bytes, int stall_us,
                                           pha_stream_t stream) {
    const pha_status st = stall_status(stall_us, dtype);
    return st != PHA_OK ? st
                        : sinks_bwd(q, k, v, o, lse, dout, cu_seqlens, batch, max_len, total_tokens, n_heads,
                                    n_kv_heads, head_dim, dtype, window, sinks, paired, scale, dq, dk, dv,
                                    workspace, workspace_bytes, stream, stall_us);
}

}  // extern "C"
