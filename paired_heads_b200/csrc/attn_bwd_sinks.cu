// attn_bwd_sinks.cu -- backward of causal attention with a sliding window and sinks on the sm_100a
// tensor cores (bf16, head_dim 64 / 128), over tile lists.
//
// Mathematics: with P recomputed from q, k and the forward's lse, and D_i = dO_i . O_i,
//   dP = dO V^T,  dS = P o (dP - D),  dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO.
// Tiles of 128 slots are counted from the document's start. Query tile j sees the key tiles of its
// window and, through the sinks (at most 128: they lie in key tile 0), key tile 0. One kernel template:
//   key-major (dK, dV): outer tile X = (K, V) of a key tile, steps Y = (Q, dO) of the query tiles that
//     see it, for every query head of the group: S^T = K Q^T, dP^T = V dO^T, dV += P^T dO,
//     dK += dS^T Q;
//   query-major (dQ): X = (Q, dO) of a query tile, steps Y = (K, V) of the key tiles it sees:
//     S = Q K^T, dP = dO V^T, dQ += dS K. Key tile 0 behind the window is a first step of as many
//     columns as there are sinks (whole K = 16 slices).
// Key tile 0 over the query tiles that only its sinks reach ("far") comes in pieces (kernels.cuh): their
// float32 rows, like the window's part of the same rows, go to p.sink_part and are summed in order by
// attn_bwd_sink_sum_kernel; so no CTA walks a whole document, and no atomics are used.
//
// What bounds it: the S and dP products read both operands from shared memory (128 bytes a clock: 64
// clocks for each K = 16 slice of a 128 x 128 product), the others one; with 16 + 16 slices that is about
// 2,050 clocks a step (key-major; 1,540 query-major), to which the chain S -> P -> dV -> S of
// one step must not add up. So the elementwise work is cut in two, P from S (stage A) and dS from dP
// (stage B), and each overlaps the other's products: while stage B runs, dV += P^T dO and the next S
// are computed; while the next stage A runs, dK += dS^T Q and the next dP. (Both stages after both
// products, as in attn_bwd_tc.cu: 798 us for dK / dV of 2 x 8192 tokens, 32 / 8 heads of 128, window
// 1024, 675 for dQ; the two column halves of a step staggered instead: 680 and 574, the halves' N = 64
// products reading X twice; this one: 530 and 367, 3,700 and 2,500 clocks a step.) What is left over the
// products' 2,050 and 1,540 clocks is the chain S -> P -> dV -> next S, P lying in S's columns. At hd 128 the
// key-major kernel has no room for a second S: S, dP, dV and dK take all 512 columns of TMEM. The query-major one spends
// its last 128 on two buffers of dS instead, and hd 64 (accumulators of 128 columns or 64) is laid out alike: there a
// second S would fit and has not been tried.
// TMEM columns: S [0, 128), dP [128, 256), accumulators from 256 (dV, dK or dQ). Key-major, P^T and dS^T
// of column half h (bf16 A operands) overwrite the first 32 of the half's own S or dP columns;
// query-major, dS goes to two buffers of 64 columns at 384 so that S and dP of the next step wait only
// for their columns to have been read.
//
// CTA = 12 warps, one per SM, persistent over the list (items dealt in snake order):
//   warps 0-7   two warpgroups, warpgroup h taking columns 64 h .. 64 h + 63 of every step (row = TMEM
//               lane) and half h of the accumulator columns in the epilogue
//   warp 8      issues the second products (dV and dK, or dQ)
//   warp 9      issues the first products (S and dP); owner of the 512 TMEM columns. (One warp for all
//               four products spent 2,500 of 5,200 clocks a step between them.) Both run as whole warps,
//               with an elected lane for the MMAs alone and a warp index that is uniform to the compiler:
//               the MMAs' operands then stay in uniform registers. (Under `if (lane == 0)` an MMA took about
//               100 clocks to issue: 637 us instead of 575 for dK / dV, 443 instead of 377 for dQ.)
//   warp 10     producer: X and Y tiles by TMA, key-major also -lse log2(e) and -D of the queries
//   warp 11     blanks the rows of a landed Y tile that lie behind the document's end: whatever is there (a
//               padded batch's NaN) would meet a zero weight, and 0 * NaN is NaN
// Every wait is bounded (1 s); on expiry the CTA records a status, drains its own copies and MMAs,
// frees TMEM and exits.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "attn_common.cuh"
#include "kernels.cuh"

namespace pha {

namespace {

constexpr int kThreads = 384;
constexpr int kRegsElementwise = 200, kRegsOther = 104;
static_assert(8 * kRegsElementwise + 4 * kRegsOther <= 12 * 168, "register split");

template <int HD, bool KEYMAJOR>
struct Layout {
    static constexpr int kChunk = 128 * 128;  // one [128 rows][64 bf16] swizzled chunk (bytes)
    static constexpr int kTile = 128 * HD * 2;
    // Buffers of Y0 and of Y1. Y0 (Q or K) is read until the step's last product and wanted first by the
    // next but one's S; Y1 (dO or V) is wanted last and done with early: with two of each, Y0 came too
    // late (1,500 clocks a step).
    static constexpr int kR0 = 3, kR1 = 1;
    static constexpr int kOffX = 0;                        // X0, X1
    static constexpr int kOffY0 = kOffX + 2 * kTile;
    static constexpr int kOffY1 = kOffY0 + kR0 * kTile;
    // key-major: per Y0 buffer -lse2[128], -D[128]; then 2 KB per warp (a 16-row box of dK / dV on its way
    // out); query-major: the dQ tile on its way out
    static constexpr int kOffVec = kOffY1 + kR1 * kTile;
    static constexpr int kOffStg = kOffVec + (KEYMAJOR ? kR0 * 2 * 128 * 4 : 0);
    static constexpr int kOffBar = kOffStg + (KEYMAJOR ? 8 * 2048 : kTile);
    static constexpr int kBarBytes = 512;
    static constexpr int kSmemBytes = kOffBar + kBarBytes + 1024;  // + slack to align to 1024
    static constexpr uint32_t kTmemCols = 512;
    static constexpr uint32_t kTmS = 0, kTmDP = 128, kTmAcc = 256, kTmDS = 384;
    static_assert(kSmemBytes <= 232448, "shared memory budget");
};

// What the producer tells the other roles, in shared memory: of each step, with its Y0 tile (read after
// y0_full or y0_ok), and of each outer tile (four of them: a step three before a tile's first one belongs
// at the latest to the tile three before it, so everybody has left the one four before). The other roles
// decode nothing: their code has to stay small beside the elementwise loops, whose instructions it pushes
// out of the cache (each role walking the list by itself, before other changes: 656 us instead of 637 for dK / dV,
// 496 instead of 441 for dQ, 2 x 8192 tokens, 32 / 8 heads of 128, window 1024).
struct StepRec {
    int flags;  // kFirst, kLast step of its outer tile; kEnd: no step, the list is done
    int y_row;  // first slot of the Y tiles
    int rows;   // rows of them inside the document
    int cols;   // columns that are multiplied
};
enum : int { kFirst = 1, kLast = 2, kEnd = 4 };
struct TileRec {
    int row0, head, doc_start, doc_end, piece;
};

struct Bars {
    uint64_t x_full, x_empty;
    uint64_t y0_full[3], y0_ok[3], y0_empty[3];
    uint64_t y1_full, y1_ok, y1_empty;
    uint64_t vec_full[3];       // key-major: -lse2 and -D of the queries
    uint64_t s_full, dp_full;   // a step's S / dP are in TMEM
    uint64_t a_done, b_done;    // stage A / B done by both warpgroups (key-major: P / dS stored; query-major,
                                // a_done: S read, b_done: dS stored)
    uint64_t dp_read;           // query-major: dP read
    uint64_t m2_done[2];        // key-major: dV's / dK's product complete (P's / dS's columns are free);
                                // query-major: dQ's of dS buffer i
    uint64_t acc_full, acc_empty, drain[2];
    uint64_t stall;             // never signalled: the failure-detection test hook waits on it
    uint32_t tmem_base;
    int abort;
    StepRec step[3];
    TileRec tile[4];
};

// The low n bits (n clamped to 0 .. 32).
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : (n >= 32 ? ~0u : (1u << n) - 1u); }

// An item of the list: its outer tile and the steps over it.
struct Tile {
    int row0;            // first slot of the outer tile
    int head;            // query head (query-major) or kv head (key-major)
    int doc_start, doc_end;
    int n_sub;           // steps
    int nq;              // key-major: query tiles per head
    int first;           // document tile of the first step's Y tile
    bool sink0;          // query-major: step 0 is key tile 0, the others follow from `first`
    int piece;           // key-major: far piece, or -1
};

template <bool KEYMAJOR>
__device__ __forceinline__ Tile decode_tile(int4 w, const AttnProblem& p, int G) {
    const BandItem it = decode_band(w);
    Tile o;
    o.row0 = it.q0;
    o.doc_start = it.doc_start;
    o.doc_end = it.doc_end;
    o.sink0 = false;
    o.piece = -1;
    const int a = it.doc_start, b = it.doc_end;
    const int j = (o.row0 - a) / kBlockN, last = (b - a - 1) / kBlockN;
    int lo, hi;
    if (!KEYMAJOR) {
        o.head = it.head;
        lo = p.window > 0 && o.row0 - p.window + 1 > a ? (o.row0 - p.window + 1 - a) / kBlockN : 0;
        hi = j;
        o.nq = 0;
        o.sink0 = p.sinks > 0 && lo > 0;
        o.n_sub = hi - lo + 1 + (o.sink0 ? 1 : 0);
    } else {
        o.head = it.head / G;
        if (it.n_qt > 1) {
            o.piece = it.n_qt - 2;
            const int c = sink_piece_tiles(p.window, p.max_len, p.slot_mult);
            lo = sink_far_tile(p.window, b - a) + o.piece * c;
            hi = min(last, lo + c - 1);
        } else {
            lo = j;
            hi = last;
            if (p.window > 0) {
                // (compared before they are added: the sum may pass 31 bits)
                const int k_last = min(o.row0 + kBlockM, b) - 1;
                hi = (k_last + min(p.window - 1, b - 1 - k_last) - a) / kBlockN;
            }
        }
        o.nq = hi - lo + 1;
        o.n_sub = G * o.nq;
    }
    o.first = lo;
    return o;
}

// Step s: the head and first slot of its Y tiles.
template <bool KEYMAJOR>
__device__ __forceinline__ void step_tile(const Tile& o, int s, int G, int& y_head, int& y_row) {
    if (KEYMAJOR) {
        y_head = o.head * G + s / o.nq;
        y_row = o.doc_start + kBlockN * (o.first + s % o.nq);
    } else {
        y_head = o.head / G;
        y_row = o.doc_start + kBlockN * (o.sink0 ? (s == 0 ? 0 : o.first + s - 1) : o.first + s);
    }
}

// Place in a ring of N buffers, and the parity of its lap.
template <int N>
struct Ring {
    uint32_t i = 0, lap = 0;
    __device__ __forceinline__ void next() {
        if (++i == N) {
            i = 0;
            lap ^= 1;
        }
    }
};

// Columns of step s that are multiplied.
template <bool KEYMAJOR>
__device__ __forceinline__ int step_cols(const Tile& o, int s, const AttnProblem& p) {
    return !KEYMAJOR && o.sink0 && s == 0 ? (p.sinks + 15) & ~15 : kBlockN;
}

template <int HD, bool KEYMAJOR>
__global__ void __launch_bounds__(kThreads, 1)
    attn_bwd_sinks_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                          const __grid_constant__ CUtensorMap tm_st, const __grid_constant__ CUtensorMap tm_st2,
                          const AttnProblem p, const float* __restrict__ nlse, const float* __restrict__ nd,
                          __nv_bfloat16* __restrict__ out_a,
                          __nv_bfloat16* __restrict__ out_b, const int4* __restrict__ items,
                          const WorkspaceHeader* hdr, int* dev_status) {
    // out_a: dQ (query-major) or dK (key-major); out_b: dV (key-major); tm_st: a map over dQ with a 64 x
    // 32 box or over dK with a 64 x 16 box; tm_st2: over dV with a 64 x 16 box (key-major)
    using L = Layout<HD, KEYMAJOR>;
    static_assert(sizeof(Bars) <= L::kBarBytes && L::kR0 <= 3 && L::kR1 == 1, "barrier block");
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_u32 = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + (((raw_u32 + 1023u) & ~1023u) - raw_u32);
    const uint32_t sbase = smem_u32(smem);
    Bars* bars = reinterpret_cast<Bars*>(smem + L::kOffBar);
    float* vec = reinterpret_cast<float*>(smem + L::kOffVec);
    volatile int* abort_flag = &bars->abort;

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);  // (uniform)
    const int lane = threadIdx.x & 31;

    if (warp == 8 && lane == 0) {
        mbar_init(&bars->x_full, 1);
        mbar_init(&bars->x_empty, 1);
        for (int s = 0; s < 3; ++s) {
            mbar_init(&bars->y0_full[s], 1);
            mbar_init(&bars->y0_ok[s], 32);
            mbar_init(&bars->y0_empty[s], 1);
            mbar_init(&bars->vec_full[s], 32);
        }
        mbar_init(&bars->y1_full, 1);
        mbar_init(&bars->y1_ok, 32);
        mbar_init(&bars->y1_empty, KEYMAJOR ? 2 : 1);  // dP's product through, and key-major dV's
        for (int s = 0; s < 2; ++s) mbar_init(&bars->m2_done[s], 1);
        mbar_init(&bars->s_full, 1);
        mbar_init(&bars->dp_full, 1);
        mbar_init(&bars->a_done, 256);
        mbar_init(&bars->b_done, 256);
        mbar_init(&bars->dp_read, 256);
        mbar_init(&bars->acc_full, 1);
        mbar_init(&bars->acc_empty, 256);
        mbar_init(&bars->drain[0], 1);
        mbar_init(&bars->drain[1], 1);
        mbar_init(&bars->stall, 1);
        bars->abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
        tma_prefetch_desc(&tm_do);
    }
    if (warp == 9) {
        tmem_alloc(&bars->tmem_base, L::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;

    const int n_items = *reinterpret_cast<const volatile int*>(&hdr->n_items);
    const int H = p.heads, Hkv = p.kv_heads, G = H / Hkv;
    // key-major: one item per kv head (that of the group's first query head)
    const int walk_g = KEYMAJOR ? G : 1;
    if (warp >= 8) regs_decrease<kRegsOther>();

    if (warp == 10) {
        // ------------------------------------------------------------ producer
        // Y = (Q, dO) (key-major) or (K, V), X the other two, by TMA. Y0 runs one step ahead of Y1: it is
        // wanted first and has more buffers.
        const CUtensorMap* mx0 = KEYMAJOR ? &tm_k : &tm_q;
        const CUtensorMap* mx1 = KEYMAJOR ? &tm_v : &tm_do;
        const CUtensorMap* my0 = KEYMAJOR ? &tm_q : &tm_k;
        const CUtensorMap* my1 = KEYMAJOR ? &tm_do : &tm_v;
        Ring<L::kR0> y0;
        uint32_t n0 = 0, n1 = 0, tiles_x = 0, tiles = 0;
        bool ok = true;
        auto acquire = [&](uint64_t* bar, uint32_t parity) {
            ok = ok && __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, dev_status));
            return ok;
        };
        // the step whose Y1 (and X, if it is a tile's first) is still to come
        bool lag = false, lag_first = false;
        int lag_head = 0, lag_row = 0, lag_x_head = 0, lag_x_row = 0;
        auto finish_lag = [&]() {
            if (!lag) return;
            if (lag_first) {
                if (!acquire(&bars->x_empty, (tiles_x & 1) ^ 1)) return;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&bars->x_full, 2 * L::kTile);
                    for (int c = 0; c < HD / 64; ++c) {
                        const int col = lag_x_head * HD + 64 * c;
                        tma_load_2d(smem + L::kOffX + c * L::kChunk, mx0, col, lag_x_row, &bars->x_full);
                        tma_load_2d(smem + L::kOffX + L::kTile + c * L::kChunk, mx1, col, lag_x_row, &bars->x_full);
                    }
                }
                ++tiles_x;
            }
            if (!acquire(&bars->y1_empty, (n1 & 1) ^ 1)) return;
            if (lane == 0) {
                mbar_arrive_expect_tx(&bars->y1_full, L::kTile);
                for (int c = 0; c < HD / 64; ++c)
                    tma_load_2d(smem + L::kOffY1 + c * L::kChunk, my1, lag_head * HD + 64 * c, lag_row, &bars->y1_full);
            }
            __syncwarp();
            ++n1;
        };
        ItemWalk wk;
        for (wk.start(items, n_items, walk_g, H); ok && !wk.done(); wk.advance()) {
            if (!wk.has()) continue;
            const Tile o = decode_tile<KEYMAJOR>(wk.cur, p, G);
            for (int s = 0; s < o.n_sub; ++s) {
                if (!acquire(&bars->y0_empty[y0.i], y0.lap ^ 1)) break;
                int y_head, y_row;
                step_tile<KEYMAJOR>(o, s, G, y_head, y_row);
                if (lane == 0) {
                    if (s == 0) bars->tile[tiles & 3] = TileRec{o.row0, o.head, o.doc_start, o.doc_end, o.piece};
                    bars->step[y0.i] = StepRec{(s == 0 ? kFirst : 0) | (s + 1 == o.n_sub ? kLast : 0), y_row,
                                               o.doc_end - y_row < kBlockN ? o.doc_end - y_row : kBlockN,
                                               step_cols<KEYMAJOR>(o, s, p)};
                    mbar_arrive_expect_tx(&bars->y0_full[y0.i], L::kTile);
                    for (int c = 0; c < HD / 64; ++c)
                        tma_load_2d(smem + L::kOffY0 + y0.i * L::kTile + c * L::kChunk, my0, y_head * HD + 64 * c, y_row,
                                    &bars->y0_full[y0.i]);
                }
                if (KEYMAJOR) {
                    // -lse * log2(e) and -D of the queries (0 past the document end), asynchronously too
                    const uint32_t to = smem_u32(vec + y0.i * 256);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int c = 32 * e + lane, qs = y_row + c;
                        const bool inside = qs < o.doc_end;
                        const int64_t r = inside ? static_cast<int64_t>(qs) * H + y_head : 0;
                        cp_async_4_zfill(to + 4 * c, nlse + r, inside ? 4u : 0u);
                        cp_async_4_zfill(to + 512 + 4 * c, nd + r, inside ? 4u : 0u);
                    }
                    cp_async_arrive(&bars->vec_full[y0.i]);
                }
                __syncwarp();
                ++n0;
                y0.next();
                finish_lag();
                lag = true;
                lag_first = s == 0;
                lag_head = y_head;
                lag_row = y_row;
                lag_x_head = o.head;
                lag_x_row = o.row0;
            }
            ++tiles;
        }
        if (ok && acquire(&bars->y0_empty[y0.i], y0.lap ^ 1)) {
            if (lane == 0) {
                bars->step[y0.i].flags = kEnd;
                mbar_arrive(&bars->y0_full[y0.i]);
            }
            __syncwarp();
            finish_lag();
        }
        cp_async_wait_all();
        if (!ok && lane == 0) {
            // Wait (bounded) for the copies issued last into every buffer.
            if (tiles_x > 0) drain_wait(&bars->x_full, (tiles_x - 1) & 1);
            if (n1 > 0) drain_wait(&bars->y1_full, (n1 - 1) & 1);
            for (uint32_t i = n0 > 3 ? n0 - 3 : 0; i < n0; ++i) drain_wait(&bars->y0_full[i % 3], (i / 3) & 1);
        }
        __syncwarp();
    } else if (warp == 11) {
        // ------------------------------------------------------------ blank rows behind the document
        Ring<L::kR0> y0;
        uint32_t n1 = 0;
        int rows = kBlockN;       // of the step whose Y1 comes next
        bool ok = true, lag = false;
        auto blank = [&](int off, int from) {
            if (from >= kBlockN) return;
            uint8_t* y = smem + off + from * 128;
            // a row is 128 bytes of each 64-column chunk (the swizzle stays inside them)
            for (int x = lane; x < (kBlockN - from) * 8; x += 32)
#pragma unroll
                for (int c = 0; c < HD / 64; ++c)
                    *reinterpret_cast<uint4*>(y + c * L::kChunk + x * 16) = make_uint4(0u, 0u, 0u, 0u);
            fence_proxy_async_smem();
        };
        for (;;) {  // (the producer's order)
            ok = __all_sync(0xffffffffu, mbar_wait(&bars->y0_full[y0.i], y0.lap, abort_flag, dev_status));
            if (!ok) break;
            const StepRec rec = bars->step[y0.i];
            const bool end = (rec.flags & kEnd) != 0;
            if (!end) blank(L::kOffY0 + y0.i * L::kTile, rec.rows);
            mbar_arrive(&bars->y0_ok[y0.i]);
            y0.next();
            if (lag) {
                ok = __all_sync(0xffffffffu, mbar_wait(&bars->y1_full, n1 & 1, abort_flag, dev_status));
                if (!ok) break;
                blank(L::kOffY1, rows);
                mbar_arrive(&bars->y1_ok);
                ++n1;
            }
            if (end) break;
            rows = rec.rows;
            lag = true;
        }
    } else if (warp == 9) {
        // ------------------------------------------------------------ the products S and dP
        constexpr uint32_t idesc = idesc_bf16_f32(kBlockM, kBlockN, 0, 0);
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, dev_status));
        };
        // d = X_w times Y (both K-major), the first `cols` columns
        auto product = [&](uint32_t d, int w, int y_off, int cols, uint64_t* full) {
            if (!ok) return;
            tc_fence_after();
            const uint32_t id = KEYMAJOR ? idesc : (idesc & ~(0x3Fu << 17)) | (static_cast<uint32_t>(cols >> 3) << 17);
            const uint64_t dx = desc_kmajor(sbase + L::kOffX + w * L::kTile, 0);
            const uint64_t dy = desc_kmajor(sbase + y_off, 0);
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < HD / 16; ++kk) {  // (as desc_kmajor steps)
                    const uint32_t step = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
                    umma_f16_ss(d, dx + step, dy + step, id, kk == 0 ? 0u : 1u);
                }
                umma_commit(full);
            }
            __syncwarp();
        };
        Ring<L::kR0> y0;
        uint32_t tiles = 0;
        for (uint32_t g = 0; ok; ++g) {
            wait(&bars->y0_ok[y0.i], y0.lap);
            if (!ok) break;
            const int flags = __shfl_sync(0xffffffffu, bars->step[y0.i].flags, 0);
            const int cols = __shfl_sync(0xffffffffu, bars->step[y0.i].cols, 0);
            if (flags & kEnd) break;
            if (flags & kFirst) {
                wait(&bars->x_full, tiles & 1);
                ++tiles;
            }
            // S, when its columns are free: key-major P lay in them (dV's product), query-major once read
            if (g > 0) wait(KEYMAJOR ? &bars->m2_done[0] : &bars->a_done, (g - 1) & 1);
            product(tmem + L::kTmS, 0, L::kOffY0 + y0.i * L::kTile, cols, &bars->s_full);
            // dP, likewise (dS lay in its columns)
            wait(&bars->y1_ok, g & 1);
            if (g > 0) wait(KEYMAJOR ? &bars->m2_done[1] : &bars->dp_read, (g - 1) & 1);
            product(tmem + L::kTmDP, 1, L::kOffY1, cols, &bars->dp_full);
            if (!ok) break;
            if (elect_one()) {
                umma_commit(&bars->y1_empty);
                if (flags & kLast) umma_commit(&bars->x_empty);
            }
            __syncwarp();
            y0.next();
        }
        // Wait (bounded) until every MMA this warp issued has finished.
        if (elect_one()) umma_commit(&bars->drain[0]);
        __syncwarp();
        drain_wait(&bars->drain[0], 0);
    } else if (warp == 8) {
        // ------------------------------------------------------------ the products dV and dK, or dQ
        constexpr uint32_t idesc = idesc_bf16_f32(kBlockM, HD, 0, 1);
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, dev_status));
        };
        // acc (+)= A (TMEM, bf16 pairs; column half h at a + h * half) times Y's rows (MN-major)
        auto product = [&](uint32_t acc, uint32_t a, uint32_t half, int y_off, bool first, int cols) {
            if (!ok) return;
            tc_fence_after();
            const uint64_t dy = desc_v(sbase + y_off, 0);
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < kBlockN / 16; ++kk) {
                    if (!KEYMAJOR && 16 * kk >= cols) continue;
                    umma_f16_ts(acc, a + (kk >> 2) * half + (kk & 3) * 8, dy + kk * (2048 >> 4), idesc,
                                (!first || kk > 0) ? 1u : 0u);
                }
            }
            __syncwarp();
        };
        Ring<L::kR0> y0;
        uint32_t tiles = 0;
        for (uint32_t g = 0; ok; ++g) {
            wait(&bars->y0_ok[y0.i], y0.lap);
            if (!ok) break;
            const int flags = __shfl_sync(0xffffffffu, bars->step[y0.i].flags, 0);
            const int cols = __shfl_sync(0xffffffffu, bars->step[y0.i].cols, 0);
            if (flags & kEnd) break;
            const bool first = (flags & kFirst) != 0;
            const int y0_off = L::kOffY0 + y0.i * L::kTile;
            wait(KEYMAJOR ? &bars->a_done : &bars->b_done, g & 1);
            if (first) {
                if (tiles > 0) wait(&bars->acc_empty, (tiles - 1) & 1);
                ++tiles;
            }
            if (KEYMAJOR) {
                wait(&bars->y1_ok, g & 1);  // (P needs S alone: dO may still be on its way)
                product(tmem + L::kTmAcc, tmem + L::kTmS, 64, L::kOffY1, first, kBlockN);
                if (!ok) break;
                if (elect_one()) {
                    umma_commit(&bars->m2_done[0]);
                    umma_commit(&bars->y1_empty);
                }
                __syncwarp();
                wait(&bars->b_done, g & 1);
                // behind the next S, which the next stage A waits for (before it: 557 us instead of 530);
                // not at a tile's end, where that S waits for X
                if (!(flags & kLast)) wait(&bars->s_full, (g + 1) & 1);
                product(tmem + L::kTmAcc + HD, tmem + L::kTmDP, 64, y0_off, first, kBlockN);
                if (!ok) break;
                if (elect_one()) umma_commit(&bars->m2_done[1]);
            } else {
                product(tmem + L::kTmAcc, tmem + L::kTmDS + 64 * (g & 1), 32, y0_off, first, cols);
                if (!ok) break;
                if (elect_one()) umma_commit(&bars->m2_done[g & 1]);
            }
            if (elect_one()) {
                umma_commit(&bars->y0_empty[y0.i]);
                if (flags & kLast) umma_commit(&bars->acc_full);
            }
            __syncwarp();
            y0.next();
        }
        if (elect_one()) umma_commit(&bars->drain[1]);
        __syncwarp();
        drain_wait(&bars->drain[1], 0);
    } else {
        // ------------------------------------------------------------ elementwise warpgroups
        regs_increase<kRegsElementwise>();
        const int h = warp >> 2;            // the column half of every step this warpgroup takes
        const int row = threadIdx.x & 127;  // TMEM lane == row of the outer tile
        const int r0 = (warp & 3) * 32;     // first row of this warp
        const uint32_t tm_lane = tmem + (static_cast<uint32_t>(r0) << 16);
        const uint64_t scale2 = f32x2(p.scale * kLog2e, p.scale * kLog2e);
        const int window = p.window;
        uint32_t oc = 0, g = 0, tiles = 0;  // outer tiles and steps done, outer tiles begun
        Ring<L::kR0> y0;
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, dev_status));
            return ok;
        };
        TileRec o{};
        uint64_t row_lse = 0, row_d = 0;  // query-major: this row's -lse * log2(e) and -D, twice
        if (p.test_stall_us > 0)  // test hook, as in the band kernel: the wait runs out, status 3, every role winds down
            mbar_wait(&bars->stall, 0, abort_flag, dev_status, 1000ull * static_cast<uint64_t>(p.test_stall_us));
        else for (;; ++g) {
            {
                if (!wait(&bars->y0_full[y0.i], y0.lap)) break;  // (its record; the tile is long there)
                const StepRec rec = bars->step[y0.i];
                if (rec.flags & kEnd) break;
                if (rec.flags & kFirst) {
                    o = bars->tile[tiles & 3];
                    ++tiles;
                    const int slot = o.row0 + row;
                    if (!KEYMAJOR && slot < o.doc_end) {
                        const int64_t r = static_cast<int64_t>(slot) * H + o.head;
                        const float l = nlse[r], d = nd[r];
                        row_lse = f32x2(l, l);
                        row_d = f32x2(d, d);
                    }
                }
                const int a = o.doc_start, b = o.doc_end, y_row = rec.y_row, n_cols = rec.cols;
                const int slot = o.row0 + row;  // key slot (key-major) or query slot
                const bool valid = slot < b;
                const uint32_t st = g & 1;
                // visible columns of this row: [c_lo, c_hi], and those below c_sk
                int c_lo, c_hi, c_sk = 0;
                if (KEYMAJOR) {  // the queries that see key `slot`
                    c_lo = slot - y_row;
                    c_hi = (window > 0 && slot - a >= p.sinks ? slot + min(window - 1, b - 1 - slot) : b - 1) - y_row;
                } else {         // the keys query `slot` sees
                    c_lo = (window > 0 ? max(a, slot - window + 1) : a) - y_row;
                    c_hi = slot - y_row;
                    c_sk = a + p.sinks - y_row;
                }
                // (a query that sees one key alone has dS = P (dP - D) = 0 exactly; the two sums, taken in different
                // orders, would leave 1e-7 where every gradient is zero)
                if (!valid || (!KEYMAJOR && (slot == a || (window == 1 && p.sinks == 0)))) c_hi = -1;
                // What nobody reads is left out: columns behind the sinks' slices in a step over them alone,
                // rows that are no sinks in a far piece (their sums are not kept).
                const bool idle = 64 * h >= n_cols || (KEYMAJOR && o.piece >= 0 && r0 >= p.sinks);
                const float* l2v = vec + y0.i * 256 + 64 * h;
                // stage A: P of the half's 64 columns, kept for stage B in registers
                float pr[64];
                if (KEYMAJOR && !wait(&bars->vec_full[y0.i], y0.lap)) break;
                if (!wait(&bars->s_full, g & 1)) break;
                tc_fence_after();
                if (!idle) {
                    uint32_t sv[64];
#pragma unroll
                    for (int cc = 0; cc < 2; ++cc) tmem_ld32(tm_lane + L::kTmS + 64 * h + 32 * cc, sv + 32 * cc);
                    tmem_wait_ld();
#pragma unroll
                    for (int cc = 0; cc < 2; ++cc) regs_after_wait(sv + 32 * cc);
                    if (!KEYMAJOR) {
                        tc_fence_before();  // S may be overwritten from here on
                        mbar_arrive(&bars->a_done);
                    }
                    // (pairs packed; the mask apart, so that tiles seen whole do not fetch its code)
#pragma unroll
                    for (int e = 0; e < 64; e += 4) {
                        ulonglong2 l4 = make_ulonglong2(row_lse, row_lse);
                        if (KEYMAJOR) l4 = *reinterpret_cast<const ulonglong2*>(l2v + e);
                        float x0, x1, x2, x3;
                        f32x2_split(fma_f32x2(f32x2(__uint_as_float(sv[e]), __uint_as_float(sv[e + 1])), scale2, l4.x), x0, x1);
                        f32x2_split(fma_f32x2(f32x2(__uint_as_float(sv[e + 2]), __uint_as_float(sv[e + 3])), scale2, l4.y), x2, x3);
                        pr[e] = ex2(x0);
                        pr[e + 1] = ex2(x1);
                        pr[e + 2] = ex2(x2);
                        pr[e + 3] = ex2(x3);
                    }
                    uint32_t bits[2];  // bit e of bits[cc]: column 64 h + 32 cc + e is visible
#pragma unroll
                    for (int cc = 0; cc < 2; ++cc) {
                        const int cb = 64 * h + 32 * cc;
                        bits[cc] = low_bits(c_hi + 1 - cb) & (~low_bits(c_lo - cb) | low_bits(c_sk - cb));
                    }
                    if (!__all_sync(0xffffffffu, (bits[0] & bits[1]) == ~0u)) {
#pragma unroll
                        for (int e = 0; e < 64; ++e) pr[e] = ((bits[e >> 5] >> (e & 31)) & 1u) ? pr[e] : 0.f;
                    }
                    if (KEYMAJOR) {
                        // P rounded to bf16 as the A operand of dV += P^T dO (stage B takes it unrounded)
                        uint32_t pk[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) pk[e] = pack_bf16x2(pr[2 * e], pr[2 * e + 1]);
                        tmem_st32(tm_lane + L::kTmS + 64 * h, pk);
                        tmem_wait_st();
                        tc_fence_before();
                        mbar_arrive(&bars->a_done);
                    }
                } else {
                    tc_fence_before();
                    mbar_arrive(&bars->a_done);
                }
                if (KEYMAJOR && h == 0 && slot == a && y_row == a) pr[0] = 0.f;  // the document's first query, likewise
                // stage B: dS = P (dP - D)
                if (!wait(&bars->dp_full, g & 1)) break;
                tc_fence_after();
                if (!idle) {
                    uint32_t dv[64];
#pragma unroll
                    for (int cc = 0; cc < 2; ++cc) tmem_ld32(tm_lane + L::kTmDP + 64 * h + 32 * cc, dv + 32 * cc);
                    tmem_wait_ld();
#pragma unroll
                    for (int cc = 0; cc < 2; ++cc) regs_after_wait(dv + 32 * cc);
                    if (!KEYMAJOR) {
                        tc_fence_before();  // dP may be overwritten from here on
                        mbar_arrive(&bars->dp_read);
                    }
                    uint32_t dk[32];
#pragma unroll
                    for (int e = 0; e < 64; e += 4) {
                        ulonglong2 d4 = make_ulonglong2(row_d, row_d);
                        if (KEYMAJOR) d4 = *reinterpret_cast<const ulonglong2*>(l2v + 128 + e);
                        float x0, x1, x2, x3;
                        f32x2_split(mul_f32x2(f32x2(pr[e], pr[e + 1]),
                                              add_f32x2(f32x2(__uint_as_float(dv[e]), __uint_as_float(dv[e + 1])), d4.x)), x0, x1);
                        f32x2_split(mul_f32x2(f32x2(pr[e + 2], pr[e + 3]),
                                              add_f32x2(f32x2(__uint_as_float(dv[e + 2]), __uint_as_float(dv[e + 3])), d4.y)), x2, x3);
                        dk[e >> 1] = pack_bf16x2(x0, x1);
                        dk[(e >> 1) + 1] = pack_bf16x2(x2, x3);
                    }
                    // query-major: the buffer's last product (two steps ago) must be through
                    if (!KEYMAJOR && g >= 2 && !wait(&bars->m2_done[st], ((g >> 1) & 1) ^ 1)) break;
                    tmem_st32(KEYMAJOR ? tm_lane + L::kTmDP + 64 * h : tm_lane + L::kTmDS + 64 * st + 32 * h, dk);
                    tmem_wait_st();
                } else if (!KEYMAJOR) {
                    mbar_arrive(&bars->dp_read);
                }
                tc_fence_before();
                mbar_arrive(&bars->b_done);
                y0.next();
                if (!(rec.flags & kLast)) continue;
            }
            // epilogue: accumulators -> bf16 rows of dQ, or of dK (scaled) and dV
            if (!wait(&bars->acc_full, oc & 1)) break;
            ++oc;
            tc_fence_after();
            const int a = o.doc_start, b = o.doc_end, slot = o.row0 + row;
            const bool valid = slot < b;
            const int out_heads = KEYMAJOR ? Hkv : H;
            const int64_t base = (static_cast<int64_t>(slot) * out_heads + o.head) * HD;
            bool store = true;  // rows of dQ, dK, dV in bf16
            if (KEYMAJOR && p.sinks > 0 && window > 0 && o.row0 == a) {
                // key tile 0: where the document has far query tiles, the sinks' rows of this part
                const int64_t slots = b - a;
                const int far = sink_far_tile(window, slots);
                if (far * static_cast<int64_t>(kBlockN) < slots) {
                    store = o.piece < 0;
                    int d = -1, z = p.batch;  // the document: last one that starts at or before
                    while (z - d > 1) {
                        const int mid = (d + z) >> 1;
                        if (static_cast<int64_t>(p.cu_seqlens[mid]) * p.slot_mult <= a) d = mid; else z = mid;
                    }
                    const int c = sink_piece_tiles(window, p.max_len, p.slot_mult);
                    const int64_t q_first = a + static_cast<int64_t>(far + o.piece * c) * kBlockN;
                    const int64_t part = o.piece < 0 ? d : p.batch + d + q_first / (static_cast<int64_t>(c) * kBlockN);
                    float* dst = p.sink_part + ((part * Hkv + o.head) * p.sinks + row) * 2 * HD;
#pragma unroll 1
                    for (int w = 0; w < 2; ++w) {
#pragma unroll 1
                        for (int cc = h * (HD / 64); cc < (h + 1) * (HD / 64); ++cc) {
                            uint32_t v[32];
                            tmem_ld32(tm_lane + L::kTmAcc + (w == 0 ? HD : 0) + 32 * cc, v);
                            tmem_wait_ld();
                            regs_after_wait(v);
                            const float mul = w == 0 ? p.scale : 1.f;
                            if (row < p.sinks)
#pragma unroll
                                for (int e = 0; e < 32; e += 4)
                                    *reinterpret_cast<float4*>(dst + w * HD + 32 * cc + e) =
                                        make_float4(__uint_as_float(v[e]) * mul, __uint_as_float(v[e + 1]) * mul,
                                                    __uint_as_float(v[e + 2]) * mul, __uint_as_float(v[e + 3]) * mul);
                        }
                    }
                }
            }
            // A warp whose 32 rows all lie inside the document (hd 128: warpgroup h owns the 64-column chunk
            // h) sends them out by TMA, dQ as one 32-row box, dK and dV 16 rows at a time through its 2 KB
            // box; otherwise every thread stores its own row.
            const bool boxes = store && HD == 128 && o.row0 + r0 + 31 < b;
#pragma unroll 1
            for (int w = 0; store && w < (KEYMAJOR ? 2 : 1); ++w) {
                // w = 0: the dS product (dQ or dK, times scale); w = 1: dV
                const uint32_t col0 = L::kTmAcc + (KEYMAJOR && w == 0 ? HD : 0);
                // (window 1 without sinks: every query sees one key alone)
                const float mul = w == 0 ? (window == 1 && p.sinks == 0 ? 0.f : p.scale) : 1.f;
                uint4 w8[HD / 16];  // this half's columns of the row
#pragma unroll
                for (int cc = 0; cc < HD / 64; ++cc) {
                    uint32_t v[32];
                    tmem_ld32(tm_lane + col0 + 32 * (h * (HD / 64) + cc), v);
                    tmem_wait_ld();
                    regs_after_wait(v);
#pragma unroll
                    for (int q4 = 0; q4 < 4; ++q4)
                        w8[4 * cc + q4] = make_uint4(
                            pack_bf16x2(__uint_as_float(v[8 * q4 + 0]) * mul, __uint_as_float(v[8 * q4 + 1]) * mul),
                            pack_bf16x2(__uint_as_float(v[8 * q4 + 2]) * mul, __uint_as_float(v[8 * q4 + 3]) * mul),
                            pack_bf16x2(__uint_as_float(v[8 * q4 + 4]) * mul, __uint_as_float(v[8 * q4 + 5]) * mul),
                            pack_bf16x2(__uint_as_float(v[8 * q4 + 6]) * mul, __uint_as_float(v[8 * q4 + 7]) * mul));
                }
                if (!boxes) {
                    __nv_bfloat16* dst = (w == 0 ? out_a : out_b) + base + h * (HD / 2);
                    if (valid)
#pragma unroll
                        for (int u = 0; u < HD / 16; ++u) *reinterpret_cast<uint4*>(dst + 8 * u) = w8[u];
                } else if (KEYMAJOR) {
                    uint8_t* stg = smem + L::kOffStg + warp * 2048;
#pragma unroll 1
                    for (int half = 0; half < 2; ++half) {
                        if ((lane >> 4) == half) {
                            const int r = lane & 15;  // row of the 16-row box
#pragma unroll
                            for (int u = 0; u < HD / 16; ++u)
                                *reinterpret_cast<uint4*>(stg + r * 128 + ((u ^ (r & 7)) << 4)) = w8[u];
                        }
                        fence_proxy_async_smem();  // the rows are read by the async proxy (TMA)
                        __syncwarp();
                        if (lane == 0) {
                            tma_store_2d(w == 0 ? &tm_st : &tm_st2, o.head * HD + 64 * h, o.row0 + r0 + 16 * half, stg);
                            tma_store_commit();
                            tma_store_wait_read();  // the box is rewritten next
                        }
                        __syncwarp();
                    }
                } else {
                    uint8_t* stg = smem + L::kOffStg + h * L::kChunk;
#pragma unroll
                    for (int u = 0; u < HD / 16; ++u)
                        *reinterpret_cast<uint4*>(stg + row * 128 + ((u ^ (row & 7)) << 4)) = w8[u];
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_2d(&tm_st, o.head * HD + 64 * h, o.row0 + r0, stg + r0 * 128);
                        tma_store_commit();
                        tma_store_wait_read();  // the staging area is rewritten by the next tile
                    }
                    __syncwarp();
                }
            }
            tc_fence_before();
            mbar_arrive(&bars->acc_empty);
        }
    }

    // ---------------------------------------------------------------- teardown
    if (warp < 8 && lane == 0) tma_store_wait_all();  // the epilogue's TMA stores have completed
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 9) tmem_dealloc(tmem, L::kTmemCols);
}

// Sum over the eight lanes of a row (in all of them); `group`: those lanes.
__device__ __forceinline__ float row_sum(float x, uint32_t group) {
#pragma unroll
    for (int s = 1; s < 8; s <<= 1) x += __shfl_xor_sync(group, x, s);
    return x;
}

// This lane's part of the dot product of two rows of bf16.
template <int N>
__device__ __forceinline__ float row_dot(const uint4 (&a)[N], const uint4 (&b)[N]) {
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int t = 0; t < N; ++t) {
        const uint32_t x[4] = {a[t].x, a[t].y, a[t].z, a[t].w}, y[4] = {b[t].x, b[t].y, b[t].z, b[t].w};
#pragma unroll
        for (int w = 0; w < 4; ++w)
            acc[w] = fmaf(__uint_as_float(x[w] << 16), __uint_as_float(y[w] << 16),
                          fmaf(__uint_as_float(x[w] & 0xFFFF0000u), __uint_as_float(y[w] & 0xFFFF0000u), acc[w]));
    }
    return (acc[0] + acc[1]) + (acc[2] + acc[3]);
}

// This lane's 16-byte units of row `row` of base [rows][HD].
template <int HD>
__device__ __forceinline__ void load_units(uint4 (&x)[HD / 64], const void* base, int64_t row) {
#pragma unroll
    for (int t = 0; t < HD / 64; ++t) x[t] = __ldg(static_cast<const uint4*>(base) + row * (HD / 8) + 8 * t + (threadIdx.x & 7));
}

// Rows that see few keys take D_i = sum_j P_ij dP_ij instead of dO_i . O_i, whose O is rounded to bf16: a
// document's first kFewKeys rows (a document of 6 tokens: dq off by 8e-3 of its norm without, 2.45e-3 with),
// and all rows where window and sinks are at most kFewWindow slots (window 6, 2 sinks: 2.6e-3 and 2.35e-3).
// Beyond, that rounding is below the one of dS itself; so many rows of 16 keys would take 190 us of 390 (32,768
// paired tokens of 6 heads of 128) for 2.5e-3 against 2.34e-3.
constexpr int kFewKeys = 16, kFewWindow = 8;

// The sum over the keys that the query of row r sees: its window's slots [win, slot] and the sinks before them,
// from the document's start `from` on. dout: the row's units; group: the eight lanes of the row.
template <int HD>
__device__ __forceinline__ float few_keys_d(const AttnProblem& p, const uint4 (&dout)[HD / 64], int64_t r, int64_t slot,
                                            int64_t from, float lse2, uint32_t group) {
    const int64_t win = p.window > 0 && slot - from >= p.window ? slot - p.window + 1 : from;
    const int n_sink = static_cast<int>(win - from < p.sinks ? win - from : p.sinks);
    const int g = static_cast<int>(r - slot * p.heads) / (p.heads / p.kv_heads), n_win = static_cast<int>(slot - win) + 1;
    uint4 q[HD / 64], k[HD / 64], v[HD / 64];
    load_units<HD>(q, p.q, r);
    float d = 0.f;
#pragma unroll 4
    for (int j = 0; j < n_win + n_sink; ++j) {
        const int64_t row = (j < n_win ? win + j : from + (j - n_win)) * p.kv_heads + g;
        load_units<HD>(k, p.k, row);
        load_units<HD>(v, p.v, row);
        const float s = row_sum(row_dot(q, k), group), dp = row_sum(row_dot(dout, v), group);
        d = fmaf(ex2(fmaf(s, p.scale * kLog2e, -lse2)), dp, d);
    }
    return d;
}

// -D_i and -lse_i log2(e) of every row (slot, head): 8 lanes per row, 16-byte loads. Reads o and dout once
// (35 us for 65,536 tokens of 6 heads, hd 128: 5.8 TB/s) and uses no work list, so it runs beside the lists'
// kernels (which take one CTA and 9 us each: 18 of 624 us for that step's training); its last block waits for
// them, so that the grid's end is theirs too. FEW: no row sees more than kFewWindow keys; otherwise a document's
// first rows have a kernel of their own (looking up every row's document here took 77 us). (cu_seqlens may be malformed here: what a row reads lies between its document's start and
// itself.)
template <int HD, bool FEW>
__global__ void __launch_bounds__(256) attn_bwd_sinks_rows_kernel(const AttnProblem p, const uint4* __restrict__ o,
                                                                  const uint4* __restrict__ dout, float* __restrict__ nlse,
                                                                  float* __restrict__ nd, int64_t rows) {
    if (!FEW) grid_dep_launch();
    const int64_t r = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) >> 3;
    const uint32_t group = 0xFFu << (threadIdx.x & 24);
    if (r < rows) {
        uint4 a[HD / 64], b[HD / 64];
        if (!FEW) load_units<HD>(a, o, r);
        load_units<HD>(b, dout, r);
        const float lse2 = p.lse[r] * kLog2e;
        float d = 0.f;
        if (!FEW) {
            d = row_sum(row_dot(a, b), group);
        } else {
            const int64_t slot = static_cast<uint32_t>(r) / static_cast<uint32_t>(p.heads);
            int doc = -1, z = p.batch;  // the last document that starts at or before the slot
            while (z - doc > 1) {
                const int mid = (doc + z) >> 1;
                if (static_cast<int64_t>(__ldg(p.cu_seqlens + mid)) * p.slot_mult <= slot) doc = mid; else z = mid;
            }
            const int64_t from = doc < 0 ? -1 : static_cast<int64_t>(__ldg(p.cu_seqlens + doc)) * p.slot_mult;
            if (from >= 0) d = few_keys_d<HD>(p, b, r, slot, from, lse2, group);
        }
        if ((threadIdx.x & 7) == 0) {
            nd[r] = -d;
            nlse[r] = -lse2;
        }
    }
    if (blockIdx.x == gridDim.x - 1) grid_dep_wait();
}

// -D of the first kFewKeys rows of every document, over what the kernel above (at the same time) writes there:
// block (document, head).
template <int HD>
__global__ void __launch_bounds__(8 * kFewKeys) attn_bwd_sinks_starts_kernel(const AttnProblem p, const uint4* __restrict__ dout,
                                                                             float* __restrict__ nd) {
    const int64_t slots = static_cast<int64_t>(p.total_tokens) * p.slot_mult;
    const int64_t from = static_cast<int64_t>(__ldg(p.cu_seqlens + blockIdx.x)) * p.slot_mult;
    const int64_t to = static_cast<int64_t>(__ldg(p.cu_seqlens + blockIdx.x + 1)) * p.slot_mult;
    const int64_t slot = from + (threadIdx.x >> 3), r = slot * p.heads + blockIdx.y;
    const bool row = from >= 0 && slot < to && slot < slots;
    float d = 0.f;
    if (row) {
        uint4 b[HD / 64];
        load_units<HD>(b, dout, r);
        d = few_keys_d<HD>(p, b, r, slot, from, p.lse[r] * kLog2e, 0xFFu << (threadIdx.x & 24));
    }
    grid_dep_wait();
    if (row && (threadIdx.x & 7) == 0) nd[r] = -d;
}

// Block (document, kv head, 256 of the values): the sinks' rows of dk, dv of documents with far query
// tiles, summed over the window's part and the pieces in order.
__global__ void __launch_bounds__(256) attn_bwd_sink_sum_kernel(const AttnProblem p, __nv_bfloat16* dk,
                                                                __nv_bfloat16* dv, const WorkspaceHeader* hdr,
                                                                const int* call_status) {
    if (hdr->status != DEV_OK || *call_status != DEV_OK) return;  // no list, or parts may be missing
    const int d = blockIdx.x, g = blockIdx.y, hd = p.head_dim;
    const int64_t a = static_cast<int64_t>(p.cu_seqlens[d]) * p.slot_mult;
    const int64_t slots = static_cast<int64_t>(p.cu_seqlens[d + 1]) * p.slot_mult - a;
    if (slots == 0) return;
    const int far = sink_far_tile(p.window, slots);
    const int n_far = static_cast<int>((slots + kBlockN - 1) / kBlockN) - far;
    if (n_far <= 0) return;
    const int c = sink_piece_tiles(p.window, p.max_len, p.slot_mult);
    const int pieces = (n_far + c - 1) / c;
    // pieces start exactly one piece apart: consecutive places
    const int64_t place = p.batch + d + (a + static_cast<int64_t>(far) * kBlockN) / (static_cast<int64_t>(c) * kBlockN);
    const int width = p.sinks * 2 * hd;
    const int x = blockIdx.z * 256 + threadIdx.x;
    if (x >= width) return;
    const int64_t stride = static_cast<int64_t>(p.kv_heads) * width;
    const float* rest = p.sink_part + (place * p.kv_heads + g) * width + x;
    float sum = p.sink_part[(static_cast<int64_t>(d) * p.kv_heads + g) * width + x];
#pragma unroll 8
    for (int f = 0; f < pieces; ++f) sum += rest[f * stride];
    const int m = x / (2 * hd), e = x % (2 * hd);  // (a document with far tiles has more than `sinks` rows)
    const int64_t row = ((a + m) * p.kv_heads + g) * hd;
    if (e < hd) dk[row + e] = __float2bfloat16_rn(sum);
    else dv[row + e - hd] = __float2bfloat16_rn(sum);
}

template <int HD, bool KEYMAJOR>
cudaError_t launch_one(const AttnProblem& p, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                       const CUtensorMap& tdo, const CUtensorMap& tst, const CUtensorMap& tst2, const float* nlse,
                       const float* nd, void* out_a, void* out_b, const int4* items, const WorkspaceHeader* hdr,
                       int* status, cudaStream_t stream) {
    using L = Layout<HD, KEYMAJOR>;
    int dev = 0, sms = 0;
    cudaError_t e;
    if ((e = cudaFuncSetAttribute(attn_bwd_sinks_kernel<HD, KEYMAJOR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  L::kSmemBytes)) != cudaSuccess ||
        (e = cudaGetDevice(&dev)) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
        return e;
    attn_bwd_sinks_kernel<HD, KEYMAJOR><<<sms, kThreads, L::kSmemBytes, stream>>>(
        tq, tk, tv, tdo, tst, tst2, p, nlse, nd, static_cast<__nv_bfloat16*>(out_a), static_cast<__nv_bfloat16*>(out_b),
        items, hdr, status);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_bwd_sinks_rows(const AttnProblem& p, const void* o, const void* dout, float* nlse, float* nd,
                                       cudaStream_t stream) {
    const int64_t rows = static_cast<int64_t>(p.total_tokens) * p.slot_mult * p.heads;
    const unsigned blocks = static_cast<unsigned>((rows * 8 + 255) / 256);
    const auto *a = static_cast<const uint4*>(o), *b = static_cast<const uint4*>(dout);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const bool few = p.window > 0 && p.window + p.sinks <= kFewWindow, wide = p.head_dim == 128;
    const cudaError_t e = cudaLaunchKernelEx(
        &cfg,
        wide ? (few ? attn_bwd_sinks_rows_kernel<128, true> : attn_bwd_sinks_rows_kernel<128, false>)
             : (few ? attn_bwd_sinks_rows_kernel<64, true> : attn_bwd_sinks_rows_kernel<64, false>),
        p, a, b, nlse, nd, rows);
    if (e != cudaSuccess || few) return e;
    cfg.gridDim = dim3(p.batch, p.heads);
    cfg.blockDim = dim3(8 * kFewKeys);
    return cudaLaunchKernelEx(&cfg, wide ? attn_bwd_sinks_starts_kernel<128> : attn_bwd_sinks_starts_kernel<64>, p, b, nd);
}

cudaError_t launch_attn_bwd_sinks_dq(const AttnProblem& p, const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                                     const CUtensorMap& tm_v, const CUtensorMap& tm_do, const CUtensorMap& tm_dq,
                                     const float* nlse, const float* nd, void* dq, const int4* items,
                                     const WorkspaceHeader* hdr, int* status, cudaStream_t stream) {
    if (p.head_dim == 128)
        return launch_one<128, false>(p, tm_q, tm_k, tm_v, tm_do, tm_dq, tm_dq, nlse, nd, dq, nullptr, items, hdr, status,
                                 stream);
    if (p.head_dim == 64)
        return launch_one<64, false>(p, tm_q, tm_k, tm_v, tm_do, tm_dq, tm_dq, nlse, nd, dq, nullptr, items, hdr, status,
                                 stream);
    return cudaErrorInvalidValue;
}

cudaError_t launch_attn_bwd_sinks_dkdv(const AttnProblem& p, const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                                       const CUtensorMap& tm_v, const CUtensorMap& tm_do, const CUtensorMap& tm_dk,
                                       const CUtensorMap& tm_dv, const float* nlse, const float* nd, void* dk, void* dv,
                                       const int4* items, const WorkspaceHeader* hdr, int* status,
                                       cudaStream_t stream) {
    cudaError_t e = cudaErrorInvalidValue;
    if (p.head_dim == 128)
        e = launch_one<128, true>(p, tm_q, tm_k, tm_v, tm_do, tm_dk, tm_dv, nlse, nd, dk, dv, items, hdr, status,
                              stream);
    else if (p.head_dim == 64)
        e = launch_one<64, true>(p, tm_q, tm_k, tm_v, tm_do, tm_dk, tm_dv, nlse, nd, dk, dv, items, hdr, status,
                              stream);
    if (e != cudaSuccess || p.sinks == 0) return e;
    attn_bwd_sink_sum_kernel<<<dim3(p.batch, p.kv_heads, (p.sinks * 2 * p.head_dim + 255) / 256), 256, 0, stream>>>(
        p, static_cast<__nv_bfloat16*>(dk), static_cast<__nv_bfloat16*>(dv), hdr, status);
    return cudaGetLastError();
}

}  // namespace pha
