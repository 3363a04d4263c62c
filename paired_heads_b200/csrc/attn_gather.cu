// attn_gather.cu -- bf16 attention on the sm_100a tensor cores over gathered keys: causal with a
// sliding window and sinks, keys in packed documents or in the pages of a cache.
//
// Mathematics: o = softmax(scale q k^T) v row by row over the visible key columns (gather.cuh), one
// pass with a running maximum and sum; a split of the columns leaves normalised partial rows and their
// log-sum-exp for attn_join_kernel.
//
// A work item is up to 256 rows, two sub-tiles of 128: `pack` query heads of one kv head's group times
// tile_tokens tokens. Packing the group multiplies the rows that each loaded key tile serves and lets
// a few new tokens fill the M = 128 of the MMA. The key columns come in tiles of 128, gathered row by
// row: any page size, the sinks behind the window's last column in the same tile, rows of no sequence
// filled with zeros (so that whatever lies there, NaN included, never meets a zero weight). TMA boxes
// could load contiguous runs with fewer instructions, but not pack sinks and window into one tile nor
// blank the rows past a cache's end.
//
// CTA = 12 warps, one per SM, persistent over the work list (most key tiles first, snake order):
//   warps 0-7   softmax, a warpgroup per sub-tile, thread = row = TMEM lane: the 128 scores in
//               registers, hidden ones set to -inf from a bit mask per 32 columns (chunks hidden from
//               a whole warp skip their exponentials), P (bf16) to TMEM, O rescaled there only when the
//               maximum grew by more than 2^8
//   warp 8      MMA issuer and TMEM owner: S_r = Q_r K^T, O_r += P_r V, software-pipelined over the
//               two sub-tiles (P V of the tile before, then S of this one)
//   warps 9-11  loaders: 16-byte cp.async with zero fill into the 128-byte-swizzled tiles; two copies
//               (K, V of a tile) stay in flight behind the one being issued
// Sub-tiles skip the key tiles that none of their rows sees. TMEM: S_r at 128 r, O_r at 256 + hd r;
// P_r at hd 64 apart (384 + 64 r), at hd 128 over S_r. Waits are bounded as in attn_tc.cu.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "attn_common.cuh"
#include "gather.cuh"
#include "kernels.cuh"

namespace pha {

namespace {

constexpr int kLoadWarps = 3;

// A decoded work item and what each sub-tile uses of its key tiles.
struct GItem {
    int q0, n_tok, chunk, pos0, where, tb, te, split;
    GatherCols cols;
    int ns;              // columns below it are sinks that lie in the window part
    int sf, sl;          // tiles [sf, sl] hold the sink columns
    int nr[2];           // rows of sub-tile r
    int wf[2], wl[2];    // window tiles of sub-tile r
    int first[2], last[2];  // first / last tile it uses in [tb, te); first > last: none
    __device__ __forceinline__ bool uses(int r, int t) const {
        return nr[r] > 0 && ((t >= wf[r] && t <= wl[r]) || (t >= sf && t <= sl));
    }
    __device__ __forceinline__ bool active(int r) const { return first[r] <= last[r]; }
};

// floor(row / pack) for row < 256: p_inv = ceil(65536 / pack), off by less than 1 / 256 <= 1 / pack.
__device__ __forceinline__ int div_pack(int row, int p_inv) { return (row * p_inv) >> 16; }

__device__ __forceinline__ GItem decode_gather(int4 a, int4 b, const GatherProblem& p, int p_inv) {
    GItem it;
    it.q0 = a.x;
    it.chunk = a.y >> 16;
    it.n_tok = a.y & 0xFFFF;
    it.pos0 = a.z;
    it.where = a.w;
    it.tb = b.x;
    it.te = b.y;
    it.split = b.z;
    it.cols = gather_cols(p, it.pos0, it.n_tok);
    it.ns = p.window > 0 ? p.sinks - it.cols.lo : 0;
    const bool sinks = it.cols.total > it.cols.n_w;
    it.sf = sinks ? it.cols.n_w / kBlockN : INT32_MAX;
    it.sl = sinks ? (it.cols.total - 1) / kBlockN : -1;
    const int n_rows = it.n_tok * p.pack;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        int nr = n_rows - kBlockM * r;
        nr = nr < 0 ? 0 : (nr > kBlockM ? kBlockM : nr);
        it.nr[r] = nr;
        it.first[r] = INT32_MAX;
        it.last[r] = -1;
        it.wf[r] = INT32_MAX;
        it.wl[r] = -1;
        if (nr > 0) {
            const int p_lo = it.pos0 + div_pack(kBlockM * r, p_inv);
            const int p_hi = it.pos0 + div_pack(kBlockM * r + nr - 1, p_inv);
            const int c_lo = p.window > 0 && it.ns <= 0 ? p_lo - p.window + 1 - it.cols.lo : 0;
            it.wf[r] = c_lo > 0 ? c_lo / kBlockN : 0;
            it.wl[r] = (p_hi - it.cols.lo) / kBlockN;
            const int w0 = it.wf[r] > it.tb ? it.wf[r] : it.tb, w1 = it.wl[r] < it.te ? it.wl[r] : it.te - 1;
            const int s0 = it.sf > it.tb ? it.sf : it.tb, s1 = it.sl < it.te ? it.sl : it.te - 1;
            if (s0 <= s1) {  // the sinks lie behind the window
                it.first[r] = s0;
                it.last[r] = s1;
            }
            if (w0 <= w1) {
                it.first[r] = w0 < it.first[r] ? w0 : it.first[r];
                it.last[r] = w1 > it.last[r] ? w1 : it.last[r];
            }
        }
    }
    return it;
}

// This CTA's items in snake order, the next one's words in flight.
struct GWalk {
    const int4* items;
    int n, k, idx;
    int4 a, b, na, nb;
    int nidx;
    __device__ __forceinline__ void fetch(int i, int4& x, int4& y) const {
        x = i >= 0 ? __ldg(items + 2 * static_cast<int64_t>(i)) : make_int4(0, 0, 0, 0);
        y = i >= 0 ? __ldg(items + 2 * static_cast<int64_t>(i) + 1) : make_int4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void start(const int4* it, int n_items) {
        items = it;
        n = n_items;
        k = 0;
        idx = band_item_index(0, n);
        fetch(idx, a, b);
        ahead();
    }
    __device__ __forceinline__ void ahead() {
        nidx = idx == -1 ? -1 : band_item_index(k + 1, n);
        fetch(nidx, na, nb);
    }
    __device__ __forceinline__ bool done() const { return idx == -1; }
    __device__ __forceinline__ bool has() const { return idx >= 0; }
    __device__ __forceinline__ void advance() {
        idx = nidx;
        a = na;
        b = nb;
        ++k;
        ahead();
    }
};

// A loader thread's copies: each tile is one group; the barrier of a group is signalled once two
// younger ones are on their way (or at once when the thread is about to wait for a free buffer).
struct LoadQueue {
    uint64_t* b0;
    uint64_t* b1;
    int n;
    __device__ __forceinline__ static void signal(uint64_t* bar) {
        fence_proxy_async_smem();  // the copies are read by the tensor cores (async proxy)
        mbar_arrive(bar);
    }
    __device__ __forceinline__ void push(uint64_t* bar) {
        cp_async_commit();
        if (n == 2) {
            cp_async_wait<2>();
            signal(b0);
            b0 = b1;
            b1 = bar;
        } else if (n == 1) {
            b1 = bar;
            n = 2;
        } else {
            b0 = bar;
            n = 1;
        }
    }
    __device__ __forceinline__ void flush() {
        cp_async_wait<0>();
        if (n > 0) signal(b0);
        if (n > 1) signal(b1);
        n = 0;
    }
};

// The score, or -inf where bit e of vis is clear (by a sign mask: one shift and one three-input
// logic operation).
__device__ __forceinline__ uint32_t bit_or_hidden(uint32_t score, uint32_t vis, int e) {
    const uint32_t keep = static_cast<uint32_t>(static_cast<int32_t>(vis << (31 - e)) >> 31);
    return (score & keep) | (0xFF800000u & ~keep);
}

template <int HD, bool PAGED>
__global__ void __launch_bounds__(kTcThreads, 1) attn_gather_kernel(const GatherProblem p, const int p_inv) {
    using L = TcLayout<HD>;
    constexpr bool kSepP = HD == 64;
    constexpr uint32_t kTmP = kSepP ? L::kTmO + 2 * HD : 0;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_u32 = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + (((raw_u32 + 1023u) & ~1023u) - raw_u32);
    const uint32_t sbase = smem_u32(smem);
    TcBars* bars = reinterpret_cast<TcBars*>(smem + L::kOffBar);
    volatile int* abort_flag = &bars->abort;
    int* dev_status = &p.hdr->status;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    if (warp == 8) {
        if (lane == 0) {
            for (int s = 0; s < L::kQSlots; ++s) {
                mbar_init(&bars->q_full[s], 32 * kLoadWarps);
                // freed by the commit after the sub-tile's last S and by its 4 softmax warps (the
                // epilogue stages O through the slot)
                mbar_init(&bars->q_empty[s], 5);
            }
            for (int s = 0; s < 4; ++s) {
                mbar_init(&bars->k_full[s], 32 * kLoadWarps);
                mbar_init(&bars->k_empty[s], 1);
                mbar_init(&bars->v_full[s], 32 * kLoadWarps);
                mbar_init(&bars->v_empty[s], 1);
            }
            for (int r = 0; r < 2; ++r) {
                mbar_init(&bars->s_full[r], 1);
                mbar_init(&bars->p_full[r], 128);
                mbar_init(&bars->pv_done[r], 1);
                mbar_init(&bars->o_ready[r], 1);
                mbar_init(&bars->s_free[r], 128);
            }
            mbar_init(&bars->drain, 1);
            bars->abort = 0;
            fence_mbar_init();
        }
        __syncwarp();
        tmem_alloc(&bars->tmem_base, L::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;

    grid_dep_wait();  // the work list is complete from here on
    const int n_items = *reinterpret_cast<volatile int*>(&p.hdr->n_items);
    const int H = p.heads, G = p.heads / p.kv_heads;
    static_assert(8 * kTcRegsSoftmax + 4 * kTcRegsOther <= 12 * 168, "register split");

    if (warp >= 8) regs_decrease<kTcRegsOther>();
    if (warp >= 9) {
        // ------------------------------------------------------------ loaders
        constexpr int kUnits = HD / 8;          // 16-byte units of a row
        constexpr int kRpi = 32 / kUnits;       // rows per instruction of a warp
        const int w = warp - 9;
        const int unit = lane % kUnits, row_in = lane / kUnits;
        const uint32_t unit_off = (unit >> 3) * L::kChunk;
        const __nv_bfloat16* q_all = static_cast<const __nv_bfloat16*>(p.q) + unit * 8;
        const __nv_bfloat16* k_all = static_cast<const __nv_bfloat16*>(p.k) + unit * 8;
        const __nv_bfloat16* v_all = static_cast<const __nv_bfloat16*>(p.v) + unit * 8;
        LoadQueue lq;
        lq.n = 0;
        uint32_t qc = 0, kc = 0;  // Q sub-tiles and key tiles issued
        bool ok = true;
        auto acquire = [&](uint64_t* bar, uint32_t parity) -> bool {
            if (__all_sync(0xffffffffu, mbar_probe(bar, parity))) return true;
            lq.flush();  // the consumer may need these before it frees the buffer
            return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, dev_status));
        };
        // address of this lane's unit of row `row` in a swizzled tile
        auto place = [&](uint32_t tile, int row) -> uint32_t {
            return tile + unit_off + row * 128 + (((unit & 7) ^ (row & 7)) << 4);
        };
        // the 128 rows of one tile whose pool rows are idx[kk] of lane row % 32 (negative: zeros)
        auto load_keys = [&](const __nv_bfloat16* src, uint32_t tile, const int (&idx)[4], int head) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                // 32 / kRpi row groups per 32 rows, dealt out to the warps in turn across the tile
                const int from = (w + kLoadWarps * 32 - kk * (32 / kRpi)) % kLoadWarps;
#pragma unroll 6
                for (int j = from; j < 32 / kRpi; j += kLoadWarps) {
                    const int r32 = j * kRpi + row_in;
                    const int x = __shfl_sync(0xffffffffu, idx[kk], r32);
                    const int64_t at = (static_cast<int64_t>(x < 0 ? 0 : x) * p.kv_heads + head) * HD;
                    cp_async_16_zfill(place(tile, 32 * kk + r32), src + at, x < 0 ? 0u : 16u);
                }
            }
        };
        GWalk wk;
        for (wk.start(p.items, n_items); ok && !wk.done(); wk.advance()) {
            if (!wk.has()) continue;
            const GItem it = decode_gather(wk.a, wk.b, p, p_inv);
            const int head = it.chunk * p.pack / G;
            for (int r = 0; ok && r < 2; ++r) {
                if (!it.active(r)) continue;
                const uint32_t sq = qc % L::kQSlots;
                ok = acquire(&bars->q_empty[sq], ((qc / L::kQSlots) & 1) ^ 1);
                if (!ok) break;
                const uint32_t tile = sbase + L::kOffQ + sq * L::kQSub;
                const int64_t base = (static_cast<int64_t>(it.q0) * H + it.chunk * p.pack) * HD;
#pragma unroll 4
                for (int j = w; j < kBlockM / kRpi; j += kLoadWarps) {
                    const int row = j * kRpi + row_in, rr = kBlockM * r + row;
                    const int tok = div_pack(rr, p_inv);
                    const bool in = row < it.nr[r];
                    const int64_t at = in ? base + (static_cast<int64_t>(tok) * H + (rr - tok * p.pack)) * HD : base;
                    cp_async_16_zfill(place(tile, row), q_all + at, in ? 16u : 0u);
                }
                lq.push(&bars->q_full[sq]);
                ++qc;
            }
            for (int t = it.tb; ok && t < it.te; ++t, ++kc) {
                int idx[4];
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    const int col = t * kBlockN + 32 * kk + lane;
                    idx[kk] = -1;
                    if (col < it.cols.total) {
                        const int64_t row = key_row<PAGED>(p, it.where, it.where, col_pos(it.cols, col));
                        if (row < 0 && p.status) atomicMax(p.status, DEV_BAD_PAGE);
                        idx[kk] = static_cast<int>(row);
                    }
                }
                const uint32_t sk = kc % L::kKStages, sv = kc % L::kVStages;
                ok = acquire(&bars->k_empty[sk], ((kc / L::kKStages) & 1) ^ 1);
                if (!ok) break;
                load_keys(k_all, sbase + L::kOffK + sk * L::kKV, idx, head);
                lq.push(&bars->k_full[sk]);
                ok = acquire(&bars->v_empty[sv], ((kc / L::kVStages) & 1) ^ 1);
                if (!ok) break;
                load_keys(v_all, sbase + L::kOffV + sv * L::kKV, idx, head);
                lq.push(&bars->v_full[sv]);
            }
        }
        lq.flush();
        __syncwarp();
    } else if (warp == 8) {
        // ------------------------------------------------------------ MMA issuer
        if (lane == 0) {
            constexpr uint32_t idesc_qk = idesc_bf16_f32(kBlockM, kBlockN, 0, 0);
            constexpr uint32_t idesc_pv = idesc_bf16_f32(kBlockM, HD, 0, 1);
            uint32_t qc = 0;    // Q sub-tiles of the items before the current one
            uint32_t g = 0;     // index of the current key tile in this CTA's stream
            uint32_t p_cnt[2] = {0, 0};        // P V products issued per sub-tile
            uint32_t s_cnt[2] = {0, 0};        // S products issued per sub-tile
            bool pv_open[2] = {false, false};  // hd 128: the last P V of r not yet seen complete
            // key tile g - 1 as sub-tile r used it: its S was issued, its P V not yet
            bool pend[2] = {false, false}, pend_first[2] = {false, false}, pend_last[2] = {false, false};
            bool ok = true;

            // O_r += P_r V_{g-1}; first: the sub-tile's first tile (O starts from zero), last: its last
            auto issue_pv = [&](int r, bool first, bool last) -> bool {
                if (!mbar_wait(&bars->p_full[r], p_cnt[r] & 1, abort_flag, dev_status)) return false;
                tc_fence_after();
                const uint32_t v_tile = sbase + L::kOffV + ((g - 1) % L::kVStages) * L::kKV;
                const uint32_t a_p = tmem + (kSepP ? kTmP + 64 * r : 128 * r);
#pragma unroll
                for (int kk = 0; kk < kBlockN / 16; ++kk)
                    umma_f16_ts(tmem + L::kTmO + HD * r, a_p + 8 * kk, desc_v(v_tile, kk), idesc_pv,
                                (!first || kk > 0) ? 1u : 0u);
                umma_commit(&bars->pv_done[r]);
                if (last) umma_commit(&bars->o_ready[r]);
                ++p_cnt[r];
                pv_open[r] = !kSepP;
                return true;
            };
            auto wait_v_prev = [&]() -> bool {
                const uint32_t n = g - 1;
                return mbar_wait(&bars->v_full[n % L::kVStages], (n / L::kVStages) & 1, abort_flag, dev_status);
            };

            GWalk wk;
            for (wk.start(p.items, n_items); ok && !wk.done(); wk.advance()) {
                if (!wk.has()) continue;
                const GItem it = decode_gather(wk.a, wk.b, p, p_inv);
                uint32_t q_slot[2], q_par[2];
                uint32_t n_act = 0;
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    q_slot[r] = (qc + n_act) % L::kQSlots;
                    q_par[r] = ((qc + n_act) / L::kQSlots) & 1;
                    n_act += it.active(r) ? 1 : 0;
                }
                for (int t = it.tb; t < it.te && ok; ++t, ++g) {
                    if (g > 0 && !wait_v_prev()) {
                        ok = false;
                        break;
                    }
                    // the previous item's last P V first: their epilogues free the Q slots that the
                    // loaders may be waiting for before they load this tile
                    if (t == it.tb) {
                        for (int r = 0; r < 2 && ok; ++r)
                            if (pend[r]) {
                                ok = issue_pv(r, pend_first[r], pend_last[r]);
                                pend[r] = false;
                            }
                        if (!ok) break;
                    }
                    const uint32_t sk = g % L::kKStages;
                    if (!mbar_wait(&bars->k_full[sk], (g / L::kKStages) & 1, abort_flag, dev_status)) {
                        ok = false;
                        break;
                    }
                    const uint32_t k_tile = sbase + L::kOffK + sk * L::kKV;
                    bool pv_now[2] = {false, false}, pv_first[2], pv_last[2];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        pv_now[r] = pend[r];
                        pv_first[r] = pend_first[r];
                        pv_last[r] = pend_last[r];
                        pend[r] = false;
                        if (!kSepP && pv_now[r]) {
                            if (!issue_pv(r, pv_first[r], pv_last[r])) {
                                ok = false;
                                break;
                            }
                            pv_now[r] = false;
                        }
                        if (!it.uses(r, t)) continue;
                        if (kSepP) {
                            // hd 64: S_r is free once the softmax has read its last tile
                            if (s_cnt[r] > 0 && !mbar_wait(&bars->s_free[r], (s_cnt[r] - 1) & 1,
                                                           abort_flag, dev_status)) {
                                ok = false;
                                break;
                            }
                        } else if (pv_open[r]) {
                            // hd 128: S_r overwrites the columns that P_r shares with it
                            if (!mbar_wait(&bars->pv_done[r], (p_cnt[r] - 1) & 1, abort_flag, dev_status)) {
                                ok = false;
                                break;
                            }
                            pv_open[r] = false;
                        }
                        if (t == it.first[r] &&
                            !mbar_wait(&bars->q_full[q_slot[r]], q_par[r], abort_flag, dev_status)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t q_tile = sbase + L::kOffQ + q_slot[r] * L::kQSub;
#pragma unroll
                        for (int kk = 0; kk < HD / 16; ++kk)
                            umma_f16_ss(tmem + 128 * r, desc_kmajor(q_tile, kk), desc_kmajor(k_tile, kk), idesc_qk,
                                        kk == 0 ? 0u : 1u);
                        umma_commit(&bars->s_full[r]);
                        if (t == it.last[r]) umma_commit(&bars->q_empty[q_slot[r]]);
                        ++s_cnt[r];
                        pend[r] = true;
                        pend_first[r] = t == it.first[r];
                        pend_last[r] = t == it.last[r];
                    }
                    if (!ok) break;
                    if (kSepP) {
                        for (int r = 0; r < 2 && ok; ++r)
                            if (pv_now[r]) ok = issue_pv(r, pv_first[r], pv_last[r]);
                        if (!ok) break;
                    }
                    if (g > 0) umma_commit(&bars->v_empty[(g - 1) % L::kVStages]);
                    umma_commit(&bars->k_empty[sk]);
                }
                qc += n_act;
            }
            if (ok && g > 0) {  // the last key tile's P V
                ok = wait_v_prev();
                for (int r = 0; r < 2 && ok; ++r)
                    if (pend[r]) ok = issue_pv(r, pend_first[r], pend_last[r]);
            }
            // Wait (bounded) until every MMA this thread issued has finished.
            umma_commit(&bars->drain);
            drain_wait(&bars->drain, 0);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax, sub-tile r
        regs_increase<kTcRegsSoftmax>();
        const int r = warp >> 2;
        const int row = threadIdx.x & 127;  // row of the sub-tile == TMEM lane
        const int r0 = (warp & 3) * 32;     // first row of this warp
        const uint32_t tm_lane = tmem + (static_cast<uint32_t>(r0) << 16);
        const uint32_t tm_s = tm_lane + 128 * r;
        const uint32_t tm_p = kSepP ? tm_lane + kTmP + 64 * r : tm_s;
        const uint32_t tm_o = tm_lane + L::kTmO + HD * r;
        const float scale_log2 = p.scale * kLog2e;
        const uint64_t scale2 = f32x2(scale_log2, scale_log2);
        const int64_t part_rows = static_cast<int64_t>(p.total_q) * p.mult * H;
        uint32_t s_cnt = 0, o_cnt = 0;
        uint32_t pv_seen = 0;  // hd 64: P V completions of this sub-tile awaited so far
        uint32_t q_seq = 0;    // index of the current item's first Q sub-tile in this CTA's stream
        bool ok = true;
        // the low n bits (n clamped to 0 .. 32)
        auto low_bits = [](int n) -> uint32_t { return n <= 0 ? 0u : (n >= 32 ? ~0u : (1u << n) - 1u); };
        GWalk wk;
        for (wk.start(p.items, n_items); ok && !wk.done(); wk.advance()) {
            if (!wk.has()) continue;
            const GItem it = decode_gather(wk.a, wk.b, p, p_inv);
            const int nr = r ? it.nr[1] : it.nr[0];
            const int t_first = r ? it.first[1] : it.first[0];
            const int t_last = r ? it.last[1] : it.last[0];
            const int wf = r ? it.wf[1] : it.wf[0], wl = r ? it.wl[1] : it.wl[0];
            const uint32_t my_q = q_seq + (r && it.active(0) ? 1 : 0);
            q_seq += (it.active(0) ? 1 : 0) + (it.active(1) ? 1 : 0);
            if (nr == 0) continue;
            const int rr = kBlockM * r + row;
            const int tok = div_pack(rr, p_inv);
            const bool valid = row < nr;
            const int64_t out_row = (static_cast<int64_t>(it.q0) + tok) * H + it.chunk * p.pack + (rr - tok * p.pack);
            if (t_first > t_last) {  // none of this split's columns: an empty partial row
                if (valid) p.part_lse[it.split * part_rows + out_row] = -INFINITY;
                continue;
            }
            // this row's visible columns: [c_lo, c_hi] and those below ns, of the window part, and the
            // sink columns [n_w, total)
            const int c_hi = valid ? it.pos0 + tok - it.cols.lo : -1;
            const int c_lo = p.window > 0 ? it.pos0 + tok - p.window + 1 - it.cols.lo : 0;
            const int n_w = valid ? it.cols.n_w : 0, total = valid ? it.cols.total : 0;
            // a tile needs no mask when every row sees all of it
            const int all_lo = p.window > 0 ? it.pos0 + div_pack(kBlockM * r + nr - 1, p_inv) - p.window + 1 - it.cols.lo : 0;
            const int all_hi = it.pos0 + div_pack(kBlockM * r, p_inv) - it.cols.lo;
            float m = -INFINITY, l = 0.f;
            for (int t = t_first; t <= t_last; ++t) {
                if (!((t >= wf && t <= wl) || (t >= it.sf && t <= it.sl))) continue;
                ok = __all_sync(0xffffffffu, mbar_wait(&bars->s_full[r], s_cnt & 1, abort_flag, dev_status));
                if (!ok) break;
                ++s_cnt;
                tc_fence_after();
                uint32_t v[128];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(tm_s + 32 * c, v + 32 * c);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 4; ++c) regs_after_wait(v + 32 * c);
                if (kSepP) {
                    tc_fence_before();  // S_r may be overwritten from here on
                    mbar_arrive(&bars->s_free[r]);
                }
                const int col0 = t * kBlockN;
                uint32_t live = 0xFu;  // 32-column chunks that some row of this warp sees
                if (!(all_lo <= col0 && col0 + kBlockN - 1 <= all_hi)) {
                    live = 0;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int cb = col0 + 32 * c;
                        const uint32_t seen = low_bits(c_hi + 1 - cb) & (~low_bits(c_lo - cb) | low_bits(it.ns - cb));
                        const uint32_t vis = seen | (low_bits(total - cb) & ~low_bits(n_w - cb));
                        if (__any_sync(0xffffffffu, vis != 0u)) live |= 1u << c;
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            v[32 * c + e] = bit_or_hidden(v[32 * c + e], vis, e);
                    }
                }
                float mx = -INFINITY;
#pragma unroll
                for (int c = 0; c < 4; ++c) mx = fmaxf(mx, chunk_max<kMaskNone>(v + 32 * c, 0, 0, 0));
                const float m_new = fmaxf(m, mx * scale_log2);
                // the reference stays until the maximum has grown by more than 2^8: O / l and the lse
                // are exact for any reference
                const bool rescale = m_new > m + 8.0f;
                const float alpha = rescale ? ex2(m - m_new) : 1.0f;
                if (rescale) m = m_new;
                const float neg_m = (m == -INFINITY) ? 0.f : -m;
                const uint64_t negm2 = f32x2(neg_m, neg_m);
                uint64_t sum_a = f32x2(0.f, 0.f), sum_b = f32x2(0.f, 0.f);
                uint32_t pk[32];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if ((live >> c) & 1u) {
                        chunk_exp<kMaskNone>(v + 32 * c, 0, 0, 0, scale2, negm2, sum_a, sum_b, pk + 16 * (c & 1));
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; ++e) pk[16 * (c & 1) + e] = 0u;
                    }
                    if (c == 1 && kSepP && pv_seen < s_cnt - 1) {
                        // hd 64: the last P V reads P_r and adds into O_r; it must be complete before P_r
                        // is overwritten and O_r rescaled
                        ok = __all_sync(0xffffffffu, mbar_wait(&bars->pv_done[r], pv_seen & 1, abort_flag, dev_status));
                        ++pv_seen;
                        tc_fence_after();
                    }
                    if (c & 1) {
                        tmem_st16(tm_p + 16 * (c - 1), pk);
                        tmem_st16(tm_p + 16 * c, pk + 16);
                    }
                }
                if (!ok) break;
                float s_lo, s_hi;
                f32x2_split(add_f32x2(sum_a, sum_b), s_lo, s_hi);
                l = l * alpha + (s_lo + s_hi);
                if (t > t_first && __any_sync(0xffffffffu, rescale)) {
                    uint32_t ov[HD];
#pragma unroll
                    for (int c = 0; c < HD / 32; ++c) tmem_ld32(tm_o + 32 * c, ov + 32 * c);
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < HD / 32; ++c) {
                        regs_after_wait(ov + 32 * c);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            ov[32 * c + e] = __float_as_uint(__uint_as_float(ov[32 * c + e]) * alpha);
                        tmem_st32(tm_o + 32 * c, ov + 32 * c);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&bars->p_full[r]);
            }
            if (!ok) break;
            ok = __all_sync(0xffffffffu, mbar_wait(&bars->o_ready[r], o_cnt & 1, abort_flag, dev_status));
            if (!ok) break;
            ++o_cnt;
            tc_fence_after();
            const float inv_l = l > 0.f ? 1.f / l : 0.f;
            uint32_t ov[HD];
#pragma unroll
            for (int c = 0; c < HD / 32; ++c) tmem_ld32(tm_o + 32 * c, ov + 32 * c);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < HD / 32; ++c) regs_after_wait(ov + 32 * c);
            if (p.n_splits > 1) {
                // a partial row: normalised o in float32 and log2 of its sum of exponentials
                if (valid) {
                    float4* dst = reinterpret_cast<float4*>(p.part_o + (it.split * part_rows + out_row) * HD);
#pragma unroll
                    for (int c = 0; c < HD / 4; ++c)
                        dst[c] = make_float4(__uint_as_float(ov[4 * c]) * inv_l, __uint_as_float(ov[4 * c + 1]) * inv_l,
                                             __uint_as_float(ov[4 * c + 2]) * inv_l, __uint_as_float(ov[4 * c + 3]) * inv_l);
                    p.part_lse[it.split * part_rows + out_row] = l > 0.f ? m + log2f(l) : -INFINITY;
                }
            } else {
                // O -> bf16 through this sub-tile's Q slot (its last S has completed): each warp stages
                // its 32 rows (16-byte units swizzled) and copies them out whole rows at a time; the
                // rows of a token's packed heads lie next to one another in memory
                constexpr int kUnitsO = HD / 8;
                uint8_t* stage = smem + L::kOffQ + (my_q % L::kQSlots) * L::kQSub + (warp & 3) * 32 * (HD * 2);
#pragma unroll
                for (int u = 0; u < kUnitsO; ++u) {
                    const uint32_t* w8 = ov + 8 * u;
                    *reinterpret_cast<uint4*>(stage + lane * (HD * 2) + ((u ^ (lane & (kUnitsO - 1))) << 4)) = make_uint4(
                        pack_bf16x2(__uint_as_float(w8[0]) * inv_l, __uint_as_float(w8[1]) * inv_l),
                        pack_bf16x2(__uint_as_float(w8[2]) * inv_l, __uint_as_float(w8[3]) * inv_l),
                        pack_bf16x2(__uint_as_float(w8[4]) * inv_l, __uint_as_float(w8[5]) * inv_l),
                        pack_bf16x2(__uint_as_float(w8[6]) * inv_l, __uint_as_float(w8[7]) * inv_l));
                }
                __syncwarp();
                constexpr int kRowsPerIter = 32 / kUnitsO;
#pragma unroll 4
                for (int j = 0; j < kUnitsO; ++j) {
                    const int rl = j * kRowsPerIter + lane / kUnitsO, u = lane % kUnitsO;
                    const int ro = __shfl_sync(0xffffffffu, static_cast<int>(out_row - static_cast<int64_t>(it.q0) * H), rl);
                    if (r0 + rl < nr) {
                        const uint4 w4 = *reinterpret_cast<const uint4*>(stage + rl * (HD * 2) + ((u ^ (rl & (kUnitsO - 1))) << 4));
                        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.o) +
                                             (static_cast<int64_t>(it.q0) * H + ro) * HD + u * 8;
                        *reinterpret_cast<uint4*>(dst) = w4;
                    }
                }
                if (valid && p.lse) p.lse[out_row] = (m + log2f(l)) * kLn2;
            }
            __syncwarp();
            fence_proxy_async_smem();
            if (lane == 0) mbar_arrive(&bars->q_empty[my_q % L::kQSlots]);
            tc_fence_before();
        }
    }

    // ---------------------------------------------------------------- teardown
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (threadIdx.x == 0 && bars->abort && p.status) atomicMax(p.status, DEV_TIMEOUT);
    if (warp == 8) tmem_dealloc(tmem, L::kTmemCols);
}

template <int HD, bool PAGED>
cudaError_t launch_gather_hd(const GatherProblem& p, int64_t max_items, cudaStream_t stream) {
    using L = TcLayout<HD>;
    cudaError_t e = cudaFuncSetAttribute(attn_gather_kernel<HD, PAGED>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmemBytes);
    if (e != cudaSuccess) return e;
    int dev = 0, sms = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(max_items < 1 ? 1 : (max_items < sms ? max_items : sms)));
    cfg.blockDim = dim3(kTcThreads);
    cfg.dynamicSmemBytes = L::kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_gather_kernel<HD, PAGED>, p, (65536 + p.pack - 1) / p.pack);
}

}  // namespace

cudaError_t launch_attn_gather(const GatherProblem& p, int64_t max_items, cudaStream_t stream) {
    if (p.head_dim == 128)
        return p.kv_lens ? launch_gather_hd<128, true>(p, max_items, stream)
                         : launch_gather_hd<128, false>(p, max_items, stream);
    if (p.head_dim == 64)
        return p.kv_lens ? launch_gather_hd<64, true>(p, max_items, stream)
                         : launch_gather_hd<64, false>(p, max_items, stream);
    return cudaErrorInvalidValue;
}

}  // namespace pha
